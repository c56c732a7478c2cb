"""The calibrated cache's descriptor follows what its fields hold, also where an address stays the same."""
import dataclasses

import pytest

torch = pytest.importorskip("torch")

from int2_rotated_kv_gb300 import pages


def _cache():
    pp = pages.plan([64] * 4, 4, 64, growth=64, all_pages=True)
    r = torch.zeros(2, 64, 64)
    return pages.allocate(pp, hkv=2, hq=4, d=64, sink=4, window=64, device="cpu", r_k=r, r_v=r,
                          clip_k=torch.ones(2), clip_v=torch.ones(2))


def _fresh(cache):
    """What a cache without a past says of the same fields."""
    d = dataclasses.replace(cache).desc()
    return [getattr(d, name) for name, _ in d._fields_]


CHANGES = {
    "num_kv_heads": lambda c: 1, "num_q_heads": lambda c: 8, "head_dim": lambda c: 128, "sink": lambda c: 0,
    "window": lambda c: 128, "code_bits": lambda c: 4,
    "int2_pool": lambda c: c.int2_pool[:c.int2_pool.numel() // 2],
    "bf16_pool": lambda c: c.bf16_pool[:c.bf16_pool.numel() // 2],
    "int2_page_table": lambda c: c.int2_page_table.view(8, 4),
    "bf16_page_table": lambda c: c.bf16_page_table.view(8, 4),
    "r_k": lambda c: c.r_k.clone(), "clip_v": lambda c: c.clip_v.clone(), "status": lambda c: None,
}


@pytest.mark.parametrize("name", CHANGES)
def test_a_changed_field_shows(name):
    c = _cache()
    assert c.bf16_page_table.shape == (4, 8)
    first = c.desc()
    before = [getattr(first, f) for f, _ in first._fields_]
    assert before == _fresh(c)
    setattr(c, name, CHANGES[name](c))
    now = c.desc()
    assert [getattr(now, f) for f, _ in now._fields_] == _fresh(c)
    assert name == "int2_page_table" or _fresh(c) != before   # (the row length is the other table's)
    assert c.desc() is now                                    # and is not made again for nothing


def test_a_tensor_resized_in_place_shows():
    c = _cache()
    c.desc()
    where = c.bf16_page_table.data_ptr(), c.bf16_pool.data_ptr()
    c.bf16_page_table.resize_(8, 4), c.bf16_pool.resize_(c.bf16_pool.numel() // 4)
    assert where == (c.bf16_page_table.data_ptr(), c.bf16_pool.data_ptr())
    d = c.desc()
    assert (d.max_pages_per_seq, d.num_bf16_pages) == (4, c.bf16_pool.numel() // (2 * 32 * 64))

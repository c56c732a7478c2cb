"""Numbers that the library takes as int32 are refused beyond that range by the binding, where
ctypes would keep their low 32 bits: 2^32 as max_new would place nothing, and report nothing."""
import numpy as np
import pytest


def test_phases_refuse_wide_numbers():
    from int2_rotated_kv_gb300 import oscar as L
    with pytest.raises(ValueError):
        L.oscar_rope_phases(1e6, (1 << 32) + 64)
    with pytest.raises(ValueError):
        L.oscar_rope_phases(1e6, 64, 2.0, (1 << 32) + 4096)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [1 << 32, (1 << 32) + 64, 1 << 31, -(1 << 32)])
def test_device_calls_refuse_wide_numbers(wide):
    import gpu_harness as H
    import kv8_harness as K
    from oracle import kv8
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 1, 2, 64, kv8.INT8, 64)
    s.place([20, 30])
    k, v = (H.bf16_tensor(x) for x in K.draw(s.rng, 4, 1, 64))
    q = H.bf16_tensor(K.queries(s.rng, 2, 1, 2, 64)[:, 0])
    lens, starts, ws = s.i32(s.lens), s.i32([0, 2, 4]), t.zeros(1 << 20, dtype=t.uint8, device=H.DEV)
    i = s.i32([0, 0])
    calls = [lambda: L.oscar_kv8_place(s.cache, k, v, lens, starts, wide),
             lambda: L.oscar_kv8_gather(s.cache, lens, i, starts, wide, k, v),
             lambda: L.oscar_kv8_attention(s.cache, q, lens, wide, t.empty_like(q), ws),
             lambda: L.oscar_kv8_workspace_size(s.cache, wide, 1, 64),
             lambda: L.oscar_kv8_workspace_size(s.cache, 2, wide, 64),
             lambda: L.oscar_kv8_workspace_size(s.cache, 2, 1, wide),
             lambda: L.oscar_extend_pages(s.cache.page_table, lens, i, s.i32([]), s.i32([0]), s.i32([0, 0]),
                                          s.i32([0] * 3), s.i32([0] * 3), s.i32([]), s.i32([]), hold_back=wide)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    s.check_pools()

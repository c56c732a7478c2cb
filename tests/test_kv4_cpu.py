"""The calls of the 4-bit cache and oscar_gather on the host: refusals before any launch, workspace
sizes."""
import ctypes

import pytest

from int2_rotated_kv_gb300 import build as build_mod
from int2_rotated_kv_gb300 import pages


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(build_mod.LIB):
        build_mod.build()
    from int2_rotated_kv_gb300 import _lib
    _lib.lib()
    return _lib


def _desc(L, **kw):
    base = dict(num_kv_heads=2, num_q_heads=6, head_dim=64, max_pages_per_seq=8, num_pages=8,
                num_tails=2, pool=256, tail=512, page_table=1024, tail_ids=None, status=None)
    base.update(kw)
    return L.Kv4Desc(**base)


BAD_DESCS = [(dict(head_dim=96), -2), (dict(num_q_heads=5), -1), (dict(num_kv_heads=0), -1),
             (dict(num_pages=0), -1), (dict(num_tails=0), -1), (dict(max_pages_per_seq=0), -1),
             (dict(pool=None), -1), (dict(pool=264), -1), (dict(tail=None), -1), (dict(tail=520), -1),
             (dict(page_table=None), -1)]


def test_descriptor_refusals(L):
    lib = L.lib()
    for bad, want in BAD_DESCS:
        d = ctypes.byref(_desc(L, **bad))
        assert lib.oscar_kv4_attention(d, 4096, 4096, None, 1, 1, 16, 4096, 4096, 1 << 20, None) == want, bad
        assert lib.oscar_kv4_place(d, 4096, 4096, 128, 128, 4096, 4096, 1, 4, 4, None) == want
        assert lib.oscar_kv4_gather(d, 4096, 4096, 4096, 1, 4, 4, 4096, 4096, None) == want
        assert lib.oscar_kv4_workspace_size(d, 1, 1, 16) == 0
    assert lib.oscar_kv4_attention(None, 4096, 4096, None, 1, 1, 16, 4096, 4096, 1 << 20, None) == -1
    assert lib.oscar_kv4_place(None, 4096, 4096, 128, 128, 4096, 4096, 1, 4, 4, None) == -1
    assert lib.oscar_kv4_gather(None, 4096, 4096, 4096, 1, 4, 4, 4096, 4096, None) == -1
    assert lib.oscar_kv4_workspace_size(None, 1, 1, 16) == 0


def test_attention_refusals(L):
    lib, d = L.lib(), ctypes.byref(_desc(L))

    def call(q=4096, lens=4096, pos=None, batch=1, rows=1, max_len=128, out=4096, ws=4096, size=8):
        return lib.oscar_kv4_attention(d, q, lens, pos, batch, rows, max_len, out, ws, size, None)

    assert call() == -3                                    # reaches the workspace check
    for kw in (dict(q=None), dict(lens=None), dict(out=None), dict(ws=None), dict(q=4104),
               dict(out=4104), dict(ws=4100), dict(batch=-1), dict(rows=-1), dict(rows=2),
               dict(max_len=0), dict(max_len=8 * 16 + 16)):
        assert call(**kw) == -1, kw
    assert call(max_len=8 * 16 + 15) == -3                 # 8 pages and a full tail
    assert call(batch=0) == 0 and call(rows=0) == 0
    assert call(batch=1 << 30, rows=4, pos=4096) == -2     # more units than a grid has
    for bad in ((0, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, (1 << 30) + 1)):
        assert lib.oscar_kv4_workspace_size(d, *bad) == 0
    # a workspace serves every smaller call
    big = ctypes.byref(_desc(L, max_pages_per_seq=8192))
    sizes = [(b, m, n) for b in (1, 5, 64, 300) for m in (1, 3, 5, 17, 90) for n in (1, 500, 9000, 131072)]
    got = {s: lib.oscar_kv4_workspace_size(big, *s) for s in sizes}
    assert all(v > 0 for v in got.values())
    for x in sizes:
        for y in sizes:
            if all(i <= j for i, j in zip(x, y)):
                assert got[x] <= got[y], (x, y)


def test_place_and_gather_refusals(L):
    lib, d = L.lib(), ctypes.byref(_desc(L))

    def place(k=4096, v=4096, ks=128, vs=128, lens=4096, starts=4096, batch=1, rows=4, new=4):
        return lib.oscar_kv4_place(d, k, v, ks, vs, lens, starts, batch, rows, new, None)

    for kw in (dict(k=None), dict(v=None), dict(k=4104), dict(v=4100), dict(ks=120), dict(vs=132),
               dict(lens=None), dict(starts=None), dict(batch=-1), dict(rows=-1), dict(new=-1)):
        assert place(**kw) == -1, kw
    assert place(batch=0) == 0 and place(rows=0) == 0 and place(new=0) == 0
    assert place(rows=1 << 31) == -2 and place(batch=1 << 20, new=1 << 20) == -2

    def gather(lens=4096, first=4096, starts=4096, batch=1, rows=4, most=4, k=4096, v=4096):
        return lib.oscar_kv4_gather(d, lens, first, starts, batch, rows, most, k, v, None)

    for kw in (dict(lens=None), dict(first=None), dict(starts=None), dict(k=None), dict(v=None),
               dict(k=4104), dict(batch=-2), dict(rows=-1), dict(most=-1)):
        assert gather(**kw) == -1, kw
    assert gather(batch=0) == 0 and gather(rows=0) == 0 and gather(most=0) == 0
    assert gather(rows=1 << 31) == -2 and gather(batch=1 << 20, most=1 << 20) == -2


def test_gather_of_the_calibrated_cache_refusals(L):
    lib = L.lib()

    def call(lens=4096, first=4096, starts=4096, batch=1, rows=4, most=4, k=4096, v=4096, **kw):
        base = dict(num_kv_heads=2, num_q_heads=4, head_dim=64, sink=4, window=64, max_pages_per_seq=4,
                    num_int2_pages=3, num_bf16_pages=3, int2_pool=256, bf16_pool=512, int2_page_table=64,
                    bf16_page_table=64, r_k=1024, r_v=1024, clip_k=64, clip_v=64, status=None, code_bits=2)
        base.update(kw)
        return lib.oscar_gather(ctypes.byref(L.CacheDesc(**base)), lens, first, starts, batch, rows, most, k, v,
                                None)

    for kw in (dict(lens=None), dict(first=None), dict(starts=None), dict(k=None), dict(v=None), dict(k=4104),
               dict(v=4100), dict(batch=-1), dict(rows=-1), dict(most=-1), dict(int2_pool=None),
               dict(bf16_pool=None), dict(int2_page_table=None), dict(bf16_page_table=None), dict(r_k=None),
               dict(r_v=1028), dict(window=0), dict(num_int2_pages=0)):
        assert call(**kw) == -1, kw
    assert call(batch=0) == 0 and call(rows=0) == 0 and call(most=0) == 0
    for kw in (dict(rows=1 << 31), dict(batch=1 << 20, most=1 << 20), dict(head_dim=96), dict(code_bits=3)):
        assert call(**kw) == -2, kw
    assert lib.oscar_gather(None, 64, 64, 64, 1, 4, 4, 64, 64, None) == -1


def test_binding_refuses_what_it_can_see(L):
    torch = pytest.importorskip("torch")
    c = pages.allocate_kv4(3, 2, 4, hkv=2, hq=4, d=64, device="cpu")
    assert c.pool.shape == (3, 2, 18 * 64 + 16) and pages.kv4_bytes_per_page(2, 64) * 3 == c.pool.numel()
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.desc()                                            # not on a CUDA device
    with pytest.raises(ValueError):
        L.oscar_kv4_place(c, x, x, i[:1], i, 1)
    c8 = pages.allocate_kv8(3, 2, 4, hkv=2, hq=4, d=64, device="cpu")
    for call in (lambda: L.oscar_kv4_place(c8, x, x, i[:1], i, 1),
                 lambda: L.oscar_kv4_gather(c8, i[:1], i[:1], i, 1, x, x),
                 lambda: L.oscar_kv4_attention(c8, x, i[:1], 16, x, x),
                 lambda: L.oscar_kv4_workspace_size(c8, 1, 1, 16),
                 lambda: L.oscar_kv8_place(c, x, x, i[:1], i, 1),
                 lambda: L.oscar_kv8_attention(c, x, i[:1], 16, x, x)):
        with pytest.raises(ValueError, match="cache must be a Kv"):
            call()


def test_gather_needs_both_pools(L):
    for pools in ((None, 1), (1, None)):
        cache = L.Cache(2, 2, 64, 4, 64, *pools, None, None, None, None, None, None)
        with pytest.raises(ValueError):
            L.oscar_gather(cache, None, None, None, 1, None, None)

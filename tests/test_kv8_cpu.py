"""The 8-bit cache, page-table and rotary calls on the host: refusals before any
launch, workspace sizes, and the rotary frequencies."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from int2_rotated_kv_gb300 import build as build_mod


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
                num_tails=2, pool=256, tail=512, page_table=1024, tail_ids=None, status=None,
                format=0)
    base.update(kw)
    return L.Kv8Desc(**base)


BAD_DESCS = [(dict(head_dim=96), -2), (dict(format=2), -2), (dict(num_q_heads=5), -1),
             (dict(num_kv_heads=0), -1), (dict(num_pages=0), -1), (dict(num_tails=0), -1),
             (dict(max_pages_per_seq=0), -1), (dict(pool=None), -1), (dict(pool=264), -1),
             (dict(tail=None), -1), (dict(tail=520), -1), (dict(page_table=None), -1)]


def test_descriptor_refusals(L):
    lib = L.lib()
    for bad, want in BAD_DESCS:
        d = ctypes.byref(_desc(L, **bad))
        assert lib.oscar_kv8_attention(d, 4096, 4096, None, 1, 1, 16, 4096, 4096, 1 << 20, None) == want, bad
        assert lib.oscar_kv8_place(d, 4096, 4096, 128, 128, 4096, 4096, 1, 4, 4, None) == want
        assert lib.oscar_kv8_gather(d, 4096, 4096, 4096, 1, 4, 4, 4096, 4096, None) == want
        assert lib.oscar_kv8_workspace_size(d, 1, 1, 16) == 0
    assert lib.oscar_kv8_attention(None, 4096, 4096, None, 1, 1, 16, 4096, 4096, 1 << 20, None) == -1


def test_attention_refusals(L):
    lib, d = L.lib(), ctypes.byref(_desc(L))

    def call(q=4096, lens=4096, pos=None, batch=1, rows=1, max_len=128, out=4096, ws=4096, size=8):
        return lib.oscar_kv8_attention(d, q, lens, pos, batch, rows, max_len, out, ws, size, None)

    assert call() == -3                                    # reaches the workspace check
    for kw in (dict(q=None), dict(lens=None), dict(out=None), dict(ws=None), dict(q=4104),
               dict(out=4104), dict(ws=4100), dict(batch=-1), dict(rows=-1), dict(rows=2),
               dict(max_len=0), dict(max_len=8 * 16 + 16)):
        assert call(**kw) == -1, kw
    assert call(max_len=8 * 16 + 15) == -3                 # 8 pages and a full tail
    assert call(batch=0) == 0 and call(rows=0) == 0
    assert call(batch=1 << 30, rows=4, pos=4096) == -2     # more units than a grid has
    one = lib.oscar_kv8_workspace_size(d, 1, 1, 128)
    assert 0 < one
    big = _desc(L, max_pages_per_seq=8192)
    sizes = [lib.oscar_kv8_workspace_size(ctypes.byref(big), b, 1, 131072) for b in (1, 64, 4096)]
    assert sizes[0] == sizes[1] == sizes[2] > one          # per resident CTA, not per sequence
    for bad in ((0, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, (1 << 30) + 1)):
        assert lib.oscar_kv8_workspace_size(d, *bad) == 0
    d = ctypes.byref(_desc(L, max_pages_per_seq=1 << 27))
    assert call(max_len=1 << 30) == -3 and call(max_len=(1 << 30) + 1) == -2


def test_place_and_gather_refusals(L):
    lib, d = L.lib(), ctypes.byref(_desc(L))

    def place(k=4096, v=4096, ks=128, vs=128, lens=4096, starts=4096, batch=1, rows=4, new=4):
        return lib.oscar_kv8_place(d, k, v, ks, vs, lens, starts, batch, rows, new, None)

    for kw in (dict(k=None), dict(v=None), dict(k=4104), dict(v=4100), dict(ks=120), dict(vs=132),
               dict(lens=None), dict(starts=None), dict(batch=-1), dict(rows=-1), dict(new=-1)):
        assert place(**kw) == -1, kw
    assert place(batch=0) == 0 and place(rows=0) == 0 and place(new=0) == 0
    assert place(rows=1 << 31) == -2 and place(batch=1 << 20, new=1 << 20) == -2

    def gather(lens=4096, first=4096, starts=4096, batch=1, rows=4, most=4, k=4096, v=4096):
        return lib.oscar_kv8_gather(d, lens, first, starts, batch, rows, most, k, v, None)

    for kw in (dict(lens=None), dict(first=None), dict(starts=None), dict(k=None), dict(v=None),
               dict(k=4104), dict(batch=-2), dict(rows=-1), dict(most=-1)):
        assert gather(**kw) == -1, kw
    assert gather(batch=0) == 0 and gather(rows=0) == 0


def test_extend_refusals(L):
    lib = L.lib()

    def call(table=4096, maxp=4, lens=4096, new=4096, batch=1, hold=0, free=4096, n_free=4,
             cursor=4096, after=4096, ps=4096, rs=4096, ids=4096, pos=4096, rows=4):
        return lib.oscar_extend_pages(table, maxp, lens, new, batch, hold, free, n_free, cursor,
                                      after, ps, rs, ids, pos, None, rows, None, None)

    for kw in (dict(table=None), dict(maxp=0), dict(lens=None), dict(new=None), dict(batch=-1),
               dict(hold=-1), dict(free=None), dict(n_free=-1), dict(cursor=None), dict(after=None),
               dict(ps=None), dict(rs=None), dict(ids=None), dict(pos=None), dict(rows=-1)):
        assert call(**kw) == -1, kw
    assert call(batch=0) == 0
    assert call(rows=1 << 31) == -2 and call(n_free=1 << 31) == -2


def test_rope_refusals(L):
    lib = L.lib()

    def call(q=4096, k=4096, pos=4096, ph=4096, n=2, hq=4, hk=1, d=64, rd=64, inter=0, amp=1.0,
             inv=0, qs=256, ks=64, qos=256, kos=64, qo=8192, ko=8192):
        return lib.oscar_rope(q, k, pos, ph, n, hq, hk, d, rd, inter, amp, inv, qs, ks, qos, kos,
                              qo, ko, None)

    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None),
               dict(ph=None), dict(n=-1), dict(hq=-1), dict(hq=0, hk=0), dict(d=1), dict(rd=0),
               dict(rd=63), dict(rd=66), dict(inter=2), dict(inv=2), dict(amp=float("nan")),
               dict(qs=255), dict(ks=63), dict(qos=255), dict(kos=63), dict(qo=4096, qos=264),
               dict(ko=4096, kos=72)):
        assert call(**kw) == -1, kw
    assert call(n=0) == 0
    assert call(d=2048, rd=64, qs=8192, ks=2048, qos=8192, kos=2048) == -2


def _turns(base, rd, i):
    """base^(-2i/rd) / (2 pi) in the host's extended precision."""
    f = np.longdouble(base) ** (np.longdouble(-2 * i) / rd)
    return f / (2 * np.longdouble("3.14159265358979323846264338327950288"))


def test_rope_phases(L):
    """Each word is the frequency times 2^64, rounded to an integer, of fp64 steps: the
    exponent -2i/rd rounded (times ln(base) < 14: 14 * 2^-53), pow, two quotients."""
    def near(words, want, rel=2.0 ** -48):
        for g, w in zip(words, want):
            w = Fraction(float(w)) * (1 << 64)
            assert abs(int(g) - w) <= Fraction(1, 2) + w * Fraction(rel), (g, float(w))
        return True

    plain = [_turns(1e6, 128, i) for i in range(64)]
    assert near(L.oscar_rope_phases(1e6, 128), plain)
    assert near(L.oscar_rope_phases(1e4, 10, 8.0), [_turns(1e4, 10, i) / 8 for i in range(5)])
    parts = []
    for f in plain:
        keep = min(max((f * 4096 - 1) / 31, 0), 1)
        parts.append((1 - keep) * f / 16 + keep * f)
    words = L.oscar_rope_phases(1e6, 128, 16.0, 4096)
    # keep f + (1 - keep) f / 16: keep is off by 2^-48 (turns / 31) at most, times f
    assert near(words, parts, 2.0 ** -43)
    assert words[0] == L.oscar_rope_phases(1e6, 128)[0]
    for bad in ((1.0, 64), (float("nan"), 64), (1e6, 0), (1e6, 7), (1e6, 64, 0.5), (1e6, 64, float("inf")),
                (1e6, 64, 2.0, -1), (1e6, 64, 2.0, 100, 5.0, 5.0), (1e6, 64, 2.0, 100, 1.0, float("nan"))):
        with pytest.raises(L.OscarError):
            L.oscar_rope_phases(*bad)


def test_binding_checks_its_tensors(L):
    """CPU tensors, types and shapes are refused before the library is entered."""
    import torch
    from int2_rotated_kv_gb300 import pages
    cache = pages.allocate_kv8(4, 2, 2, hkv=1, hq=2, d=64, device="cpu")
    assert cache.pool.numel() == 4 * pages.kv8_bytes_per_page(1, 64)
    with pytest.raises(ValueError):
        L.oscar_kv8_workspace_size(cache, 1, 1, 16)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.oscar_rope(x, None, torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.oscar_extend_pages(torch.zeros(2, 2, dtype=torch.int32), i, i, i, i, i, i, i, i, i)

"""One workspace for a loop's calls: the size of the largest call serves every smaller one,
whichever form of the kernel that takes."""
import ctypes
import random

import numpy as np
import pytest

from int2_rotated_kv_gb300 import build as build_mod


def _lib():
    import os
    if not os.path.exists(build_mod.LIB):
        build_mod.build()
    from int2_rotated_kv_gb300 import _lib as L
    L.lib()
    return L


def test_size_covers_smaller_calls():
    L, rng = _lib(), random.Random(0)
    size = L.lib().oscar_kv8_workspace_size
    for _ in range(4000):
        h, g, d = rng.choice([1, 2, 3, 8]), rng.choice([1, 3, 4, 8, 40]), rng.choice([64, 128])
        desc = L.Kv8Desc(num_kv_heads=h, num_q_heads=h * g, head_dim=d, max_pages_per_seq=8192, num_pages=8,
                         num_tails=2, pool=256, tail=512, page_table=1024, tail_ids=None, status=None, format=0)
        most = [int(2 ** rng.uniform(0, x)) for x in (10, 9, 17)]
        some = [rng.choice([1, n, rng.randint(1, n)]) for n in most]
        assert 0 < size(ctypes.byref(desc), *some) <= size(ctypes.byref(desc), *most), (h, g, d, most, some)


@pytest.mark.gpu
def test_smaller_calls_with_the_workspace_of_a_larger():
    import gpu_harness as H
    import kv8_harness as K
    from oracle import kv8
    t, L = H.torch(), H.lib()
    b, most = 401, 48
    s = K.Sequences(b, 2, 8, 128, kv8.INT8, most, seed=1)
    s.place(np.random.default_rng(0).integers(1, most + 1, b))
    ws = t.empty(L.oscar_kv8_workspace_size(s.cache, b, 12, most), dtype=t.uint8, device=H.DEV)
    for batch, m, longest in ((b, 1, most), (108, 1, 44), (b, 12, most), (40, 12, 31), (3, 2, 48), (1, 12, 48)):
        lens = np.minimum(s.lens[:batch], longest)
        lens = np.where(lens < s.lens[:batch], lens // 16 * 16, lens)   # only whole pages of a shortened sequence
        q = K.queries(s.rng, batch, m, 8, 128)
        pos = None if m == 1 else np.maximum(lens[:, None] - m + np.arange(m), -1)
        got = s.attend(q, pos, max_len=longest, lens=lens, ws=ws)
        s.check_attention(got, q, pos, lens=lens, heads={(i, i % 2) for i in range(batch)})
    assert H.status(s.cache) == 0

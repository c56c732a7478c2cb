"""oscar_gather on the host: what of a cache's descriptor it asks for."""
import ctypes
import os

import pytest

from int2_rotated_kv_gb300 import build as build_mod


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(build_mod.LIB):
        build_mod.build()
    from int2_rotated_kv_gb300 import _lib
    return _lib


def test_needs_no_clips(L):
    """Clips are for storing: whoever reads may not have them.  (No rows, so that nothing is launched.)"""
    base = dict(num_kv_heads=2, num_q_heads=4, head_dim=64, sink=4, window=64, max_pages_per_seq=4,
                num_int2_pages=3, num_bf16_pages=3, int2_pool=256, bf16_pool=512, int2_page_table=64,
                bf16_page_table=64, r_k=1024, r_v=1024, clip_k=64, clip_v=64, status=None, code_bits=2)
    for change, want in (({}, 0), (dict(clip_k=None), 0), (dict(clip_k=None, clip_v=None), 0), (dict(r_k=None), -1)):
        d = ctypes.byref(L.CacheDesc(**{**base, **change}))
        assert L.lib().oscar_gather(d, 4096, 4096, 4096, 1, 0, 4, 4096, 4096, None) == want, change
        if "r_k" not in change and change:   # (storing does)
            assert L.lib().oscar_quantize_append(d, 4096, 4096, 4096, 0, None) == -1

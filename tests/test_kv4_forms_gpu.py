"""Every form of 4-bit attention (tiles of 8, 16, 24 and 128 columns; CTAs that share pages, clusters, teams), for
both head sizes: that these sizes take it, and that it is right for ragged, short and empty sequences."""
import json
import os
import re
import subprocess
import sys

import numpy as np
import pytest

import gpu_harness as H
import kv4_harness as K
import kv8_harness as K8

pytestmark = pytest.mark.gpu

BATCH = 16
SHARES, CLUSTER, TEAMS = 0, 1, 2
# tiles of 8 columns (16: the tiles of 128) and how the work is divided; KV heads, query heads of each, rows,
# pages announced
FORMS = [
    ((1, SHARES), (2, 8, 1, 4000)), ((1, CLUSTER), (2, 8, 1, 250)), ((1, TEAMS), (2, 8, 5, 20)),
    ((2, SHARES), (2, 8, 2, 4000)), ((2, SHARES), (3, 3, 3, 4000)), ((2, CLUSTER), (2, 8, 2, 250)),
    ((3, SHARES), (2, 8, 3, 4000)), ((3, CLUSTER), (2, 8, 3, 250)), ((16, SHARES), (2, 8, 5, 4000)),
]
CASES = [(d, form, sizes) for d in (64, 128) for form, sizes in FORMS]
LENS = np.array([0, 1, 15, 16, 17, 40, 333, 900, 1500, 5, 64, 65, 700, 31, 0, 1207])


@pytest.mark.parametrize("d,form,sizes", CASES)
def test_matches_oracle(d, form, sizes):
    hkv, g, m, announced = sizes
    lens = np.minimum(LENS, 16 * announced)
    s = K.Sequences(BATCH, hkv, hkv * g, d, 1520, seed=d + m, permute_tails=True)
    s.place(lens)
    q = K8.queries(s.rng, BATCH, m, hkv * g, d)
    pos = None
    if m > 1:   # the last positions; all over; rows that see nothing
        pos = np.maximum(lens[:, None] - m + np.arange(m), -1)
        pos[7] = s.rng.integers(0, lens[7], m)
        pos[12, 0] = -1
    if announced > s.max_pages:
        got = s.attend(q, pos, wide=announced)
        again = s.attend(q, pos, wide=announced)
    else:
        got, again = (s.attend(q, pos, max_len=16 * announced) for _ in range(2))
    s.check_attention(got, q, pos)
    np.testing.assert_array_equal(got, again)
    assert (got[lens == 0] == 0).all() and H.status(s.cache) == 0


def _names():
    """Names of the kernels that the cases launch (of sequences without a token), as JSON: run as a program, so that the
    profiler stays out of the tests' process."""
    import torch
    from torch.profiler import ProfilerActivity, profile

    from int2_rotated_kv_gb300 import _lib as L
    from int2_rotated_kv_gb300 import pages
    found = []
    for d, _, (hkv, g, m, announced) in [CASES[0]] + CASES:   # (the first once more: for the profiler to start)
        c = pages.allocate_kv4(4, BATCH, announced, hkv=hkv, hq=hkv * g, d=d, device="cuda:0")
        q = torch.zeros(BATCH, m, hkv * g, d, dtype=torch.bfloat16, device="cuda:0")
        q = q[:, 0].contiguous() if m == 1 else q
        i32 = dict(dtype=torch.int32, device="cuda:0")
        pos = torch.full((BATCH, m), -1, **i32) if m > 1 else None
        ws = torch.empty(L.oscar_kv4_workspace_size(c, BATCH, m, 16 * announced), dtype=torch.uint8, device="cuda:0")
        lens, out = torch.zeros(BATCH, **i32), torch.empty_like(q)
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as seen:
            L.oscar_kv4_attention(c, q, lens, 16 * announced, out, ws, q_pos=pos)
            torch.cuda.synchronize()
        found.append([e.name for e in seen.events()])
    print("NAMES" + json.dumps(found[1:]))


def test_these_sizes_take_them():
    here = os.path.dirname(os.path.abspath(__file__))
    code = f"import sys; sys.path[:0] = {[os.path.dirname(here), here]!r}; import test_kv4_forms_gpu as t; t._names()"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    found = json.loads(r.stdout.split("NAMES")[1])
    if not any(found):
        pytest.skip("the profiler shows no kernels here")
    for (d, (nt, mode), sizes), names in zip(CASES, found):
        want = rf"kv8_rows_kernel<{d}, 2>" if nt == 16 else rf"kv4_attention_kernel<{d}, {nt}, \(oscar::Kv8Mode\){mode}>"
        assert any(re.search(want, x) for x in names), (d, nt, mode, sizes, names)

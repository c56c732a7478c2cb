"""oscar_gather for batches of very different lengths: every tile is done once, by CTAs that share them evenly."""
import numpy as np
import pytest

import gpu_harness as H
from test_gather_gpu import Model

pytestmark = pytest.mark.gpu


def _microseconds(m, first, count, announced, calls=20):
    """GPU time of a call, from a graph of them."""
    t, L = H.torch(), H.lib()
    i32 = dict(dtype=t.int32, device=H.DEV)
    lens, begin = t.tensor(m.lens, **i32), t.tensor(first, **i32)
    starts = t.tensor(np.concatenate([[0], np.cumsum(count)]), **i32)
    outs = [t.empty(int(sum(count)), m.hkv, m.d, dtype=t.bfloat16, device=H.DEV) for _ in range(2)]
    L.oscar_gather(m.cache, lens, begin, starts, announced, *outs)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        for _ in range(calls):
            L.oscar_gather(m.cache, lens, begin, starts, announced, *outs)
    best = np.inf
    for _ in range(6):
        a, b = t.cuda.Event(enable_timing=True), t.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        t.cuda.synchronize()
        best = min(best, 1000 * a.elapsed_time(b) / calls)
    return best


@pytest.mark.parametrize("hkv,batch", [(8, 256), (4, 128)])
def test_short_sequences_beside_a_longer_one(hkv, batch):
    """What is announced does not decide who does the work: as many tiles a sequence as CTAs have the same
    rotation is as good as one more."""
    ctas = H.lib().lib().oscar_device_sm_count() // (2 * hkv)
    longest = 128 * ctas - 22
    lens = np.full(batch, 100)
    lens[batch // 3] = longest
    m = Model(lens, hkv, 128, 4, seed=hkv)
    first = np.zeros(batch, int)
    even = _microseconds(m, first, lens, longest + 6)      # at most `ctas` tiles each
    other = _microseconds(m, first, lens, longest + 134)   # one more
    print(f"{batch} sequences, {hkv} heads: {even:.1f} us, {other:.1f} us")
    assert even < 1.5 * other and other < 1.5 * even
    starts, outs = m.run(first, lens, max_rows=longest + 6)
    m.check(first, lens, starts, outs, heads={(0, 0), (batch // 3, hkv - 1), (batch - 1, 1)})
    assert H.status(m.cache) == 0


@pytest.mark.parametrize("hkv", [8, 4])
def test_sequences_of_as_many_tiles_as_ctas(hkv):
    """The tiles that hold a sequence's BF16 tokens, its last, do not all fall to the same CTA: a tile takes as long as
    where a sequence has one tile more."""
    ctas = H.lib().lib().oscar_device_sm_count() // (2 * hkv)
    times = []
    for tiles in (ctas, ctas + 1):
        lens = np.full(64, 128 * tiles - 20)
        m = Model(lens, hkv, 128, 2, seed=hkv)
        times.append(_microseconds(m, np.zeros(64, int), lens, int(lens[0])) / tiles)
    print(f"{hkv} heads: {times[0]:.2f} and {times[1]:.2f} us for a tile of each")
    assert times[0] < 1.3 * times[1]


@pytest.mark.parametrize("d,hkv,bits", [(64, 2, 2), (128, 8, 4), (128, 1, 2)])
def test_sequences_without_rows_among_others(d, hkv, bits):
    """Batches that pass 32 sequences, most of which ask for nothing, a few rows, or several tiles; one of them
    refused."""
    rng = np.random.default_rng(d + hkv)
    batch = 77
    lens = rng.integers(1, 60, batch)
    lens[[0, 31, 32, 70]] = 600, 1300, 129, 257
    m = Model(lens, hkv, d, bits, seed=d)
    first = rng.integers(0, lens)
    count = np.where(rng.random(batch) < 0.4, 0, rng.integers(0, lens - first + 1))
    first[31], count[31], count[32:64:3] = 5, 1295, 0
    starts, outs = m.run(first, count)
    heads = {(b, h) for b in range(batch) for h in (0, hkv - 1)}
    m.check(first, count, starts, outs, heads=heads)
    assert H.status(m.cache) == 0
    asked = m.lens.copy()
    asked[31] -= 1                                         # (its rows end behind what is said to be stored)
    _, got = m.run(first, count, lens=asked)
    L = H.lib()
    assert H.status(m.cache) == L.DEVERR_SEQ_LEN
    s = slice(starts[31], starts[32])
    for a, b in zip(got, outs):
        assert (a[s] == 7).all()
        a[s] = b[s]
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("hkv", [1, 2, 16, 38, 40, 80])
def test_every_number_of_ctas(hkv):
    """From as many CTAs a rotation as there are SM pairs to one, and more rotations than SMs; batches of one look
    and of three, of more tiles than CTAs and of fewer."""
    rng = np.random.default_rng(hkv)
    for batch, top in ((1, 900), (9, 40), (32, 300), (70, 500)):
        lens = rng.integers(1, top, batch)
        lens[batch // 2] = 2 * top
        m = Model(lens, hkv, 64, 2, seed=batch)
        first = np.where(rng.random(batch) < 0.5, 0, rng.integers(0, lens))
        count = lens - first
        starts, outs = m.run(first, count)
        m.check(first, count, starts, outs, heads={(b, h) for b in range(batch) for h in {0, hkv - 1}})
        assert H.status(m.cache) == 0

"""GPU parity of the 4-bit cache: placement byte for byte, reading back, attention of one and several
rows, against the fp64 oracle; what the calls refuse or report; and a run of them together with page
tables and rotary positions."""
import numpy as np
import pytest

import gpu_harness as H
import kv4_harness as K
import kv8_harness as K8
from int2_rotated_kv_gb300 import pages, synth
from oracle import kv4, kv8

pytestmark = pytest.mark.gpu

WIDE = [0, 131072]   # announced table: other forms of the kernel
BIG = float(synth.bf16_from_bits(np.array([0x7F7F], np.uint16))[0])


# ---------------------------------------------------------------------- placing

@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3), (128, 8), (64, 5)])
def test_placing_in_any_pieces_gives_the_same_pages(d, hkv):
    """Prompts, chunks that start and end inside pages, single tokens, sequences that rest: pages
    and tails byte for byte after every call."""
    s = K.Sequences(5, hkv, hkv, d, 140, seed=d + hkv, permute_tails=hkv == 3)
    for new in ([1, 0, 15, 16, 17], [1, 5, 1, 1, 31], [16, 11, 0, 47, 1], [13, 1, 33, 2, 0],
                [1, 1, 1, 1, 1], [20, 0, 15, 3, 40]):
        s.place(new, packed=hkv == 8)
        s.check_pools()
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_placing_every_magnitude(d):
    """Blocks from nothing beside their page to its largest, values on the ties between codes."""
    s = K.Sequences(1, 1, 1, d, 700)
    rng = np.random.default_rng(5)
    k, v = (rng.standard_normal((16 * 40, 1, d)) for _ in range(2))
    k *= np.exp2(rng.uniform(-20, 0, (1, 1, d)))                  # channels' own scales
    k *= np.exp2(rng.integers(-90, 90, (40, 1, 1))).repeat(16, 0)  # and pages'
    v *= np.exp2(rng.uniform(-20, 0, (16 * 40, 1, d // 16))).repeat(16, -1)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for x in (k, v):
        x[:16] = rng.choice(ties, (16, 1, d)) * rng.choice([-1, 1], (16, 1, d))
        x[0] = 6.0
        x[:, 0, ::16] = np.abs(x[:, 0, ::16])
        x[:16, 0, ::16] = 6.0
    k, v = (synth.bf16_round(x.astype(np.float32)) for x in (k, v))
    s.place([16 * 40], k, v)
    s.check_pools()


def test_placing_special_values():
    """Zero and tiny pages, the largest and smallest bf16 values, NaN and infinities."""
    d = 64
    s = K.Sequences(1, 1, 1, d, 200)
    k, v = K8.draw(s.rng, 16 * 9 + 5, 1, d)
    k[0:16] = 0.0
    k[16:32] = 2.0 ** -98
    k[32:48] = 2.0 ** -97
    k[48] = BIG
    v[48:64] *= np.float32(2.0 ** -90)
    v[0, 0, 0] = -BIG
    k[64, 0, 3], k[65, 0, 4], k[66, 0, 5] = np.nan, np.inf, -np.inf
    v[80:96] = np.nan
    v[96:112] = np.inf
    v[97, 0, 1] = -1e-39          # a subnormal, and nothing else that is finite
    k[112:128, 0] = np.linspace(-1, 1, 16 * d).reshape(16, d)
    v[112:128, 0, 16:32] = 0      # blocks of zeros, and of negative zeros
    v[112:128, 0, 32:48] = -0.0
    k, v = (np.where(np.isfinite(x), synth.bf16_round(np.nan_to_num(x)), x) for x in (k, v))
    k[148, 0, 0] = np.nan         # stays in the tail as it is
    s.place([16 * 9 + 5], k, v)
    s.check_pools()
    assert H.status(s.cache) == H.lib().DEVERR_NONFINITE


def test_rows_behind_the_last_sequence_and_other_streams():
    t = H.torch()
    s = K.Sequences(3, 2, 2, 128, 100)
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(stream):
        s.place([33, 0, 20], extra_rows=7)
    s.place([1, 2, 0], stream=stream, max_new=50)
    stream.synchronize()
    s.check_pools()


def test_placing_reports_what_it_skips():
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 1, 1, 64, 64)
    s.place([10, 20])
    k, v = (H.bf16_tensor(x) for x in K8.draw(s.rng, 30, 1, 64))

    def call(lens, starts, max_new):
        L.oscar_kv4_place(s.cache, k, v, s.i32(lens), s.i32(starts), max_new)
        st = H.status(s.cache)
        s.cache.status.zero_()
        return st

    assert call([10, 20], [0, 9, 9], 8) == L.DEVERR_SEQ_LEN          # more rows than max_new
    assert call([10, 20], [0, 0, 31], 64) == L.DEVERR_SEQ_LEN        # rows behind the tensors
    assert call([10, 20], [5, 0, 0], 64) == L.DEVERR_SEQ_LEN         # descending
    assert call([-1, 20], [0, 4, 4], 64) == L.DEVERR_SEQ_LEN
    assert call([70, 20], [0, 16, 16], 64) == L.DEVERR_SEQ_LEN       # behind the page table
    s.cache.page_table[0, 0] = -1
    s.cache.page_table[1, 1] = s.cache.pool.shape[0]
    assert call([0, 20], [0, 16, 28], 64) == L.DEVERR_PAGE_ID
    s.cache.page_table.copy_(t.from_numpy(s.table))
    s.cache.tail_ids = s.i32([-1, s.cache.tail.shape[0]])
    assert call([10, 20], [0, 3, 6], 64) == L.DEVERR_PAGE_ID
    s.cache.tail_ids = None
    s.check_pools()                                                   # none of it wrote anything


@pytest.mark.parametrize("d,hkv", [(64, 2), (128, 3)])
def test_gather(d, hkv):
    t, L = H.torch(), H.lib()
    s = K.Sequences(4, hkv, hkv, d, 120, seed=7)
    s.place([100, 0, 31, 64])
    first, count = np.array([3, 0, 30, 16]), np.array([97, 0, 1, 33])
    starts = np.concatenate([[0], np.cumsum(count)])
    n = starts[-1]
    ko, vo = (t.full((n + 2, hkv, d), 7.0, dtype=t.bfloat16, device=H.DEV) for _ in range(2))
    L.oscar_kv4_gather(s.cache, s.i32(s.lens), s.i32(first), s.i32(starts), 97, ko, vo)
    t.cuda.synchronize()
    for kv, out in enumerate((ko, vo)):
        got = out.float().cpu().numpy()
        assert (got[n:] == 7).all()
        for b in range(4):
            for h in range(hkv):
                y = s.stored(b, h)[kv][first[b]:first[b] + count[b]].astype(np.float32)
                np.testing.assert_array_equal(got[starts[b]:starts[b + 1], h], synth.bf16_round(y))
    assert H.status(s.cache) == 0
    ko.fill_(7.0)
    L.oscar_kv4_gather(s.cache, s.i32(s.lens), s.i32([4, 0, 0, 0]), s.i32(starts), 97, ko, vo)
    assert H.status(s.cache) == L.DEVERR_SEQ_LEN                      # 4 + 97 > 100 tokens
    assert (ko[:97] == 7).all()
    s.cache.status.zero_()
    s.cache.page_table[0, 2] = -1
    L.oscar_kv4_gather(s.cache, s.i32(s.lens), s.i32(first), s.i32(starts), 97, ko, vo)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    assert (ko[29:45] == 7).all() and not (ko[:29] == 7).all() and not (ko[45:97] == 7).all()


# -------------------------------------------------------------------- attention

@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("d,hkv,g", [(64, 1, 4), (128, 2, 1), (128, 2, 4), (64, 3, 3), (128, 1, 8),
                                     (128, 1, 16), (64, 1, 40), (128, 2, 5)])
def test_decode_matches_oracle(d, hkv, g, wide):
    """Ragged lengths, with none, one token, and ends on and beside page borders."""
    lens = [0, 1, 15, 16, 17, 33, 700, 2607, 1024]
    s = K.Sequences(len(lens), hkv, hkv * g, d, 2700, seed=g)
    s.place(lens)
    q = K8.queries(s.rng, len(lens), 1, hkv * g, d)
    got = s.attend(q, wide=wide)
    s.check_attention(got, q)
    assert (got[0] == 0).all() and H.status(s.cache) == 0
    # fewer tokens than placed pages hold: whole pages are read from the pool all the same
    short = np.array([0, 1, 15, 16, 16, 32, 688, 1600, 1008])
    s2 = s.attend(q, lens=short, wide=wide)
    for b in (4, 5, 6, 7, 8):
        one = np.zeros_like(short)
        one[b] = short[b]
        s.check_attention(s2, q, lens=one, heads={(b, h) for h in range(hkv)})


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("d,hkv,g,m", [(64, 1, 4, 2), (128, 2, 4, 3), (128, 1, 1, 11), (128, 2, 4, 9),
                                       (64, 2, 8, 5), (128, 1, 3, 37), (128, 2, 4, 5), (64, 1, 6, 8)])
def test_rows_match_oracle(d, hkv, g, m, wide):
    """Several rows: the last positions, positions all over the context in no order, rows that see
    nothing, and rows behind the end (zeros, reported)."""
    lens = [40, 0, 555, 1700]
    s = K.Sequences(4, hkv, hkv * g, d, 1800, seed=m)
    s.place(lens)
    q = K8.queries(s.rng, 4, m, hkv * g, d)
    pos = np.array([[L - m + i if L >= m else i for i in range(m)] for L in lens])
    pos[1] = -1
    pos[2] = s.rng.integers(0, 555, m)
    pos[2, 0], pos[2, 1] = 0, -5
    got = s.attend(q, pos, wide=wide)
    s.check_attention(got, q, pos)
    assert (got[1] == 0).all() and (got[2, 1] == 0).all()
    assert H.status(s.cache) == 0
    pos[3, 0] = 1700
    got = s.attend(q, pos, wide=wide)
    assert (got[3, 0] == 0).all() and H.status(s.cache) == H.lib().DEVERR_SEQ_LEN
    s.check_attention(got, q, pos)


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("d,hkv,g,m", [(128, 2, 1, 17), (64, 1, 2, 64), (128, 1, 4, 33), (128, 1, 2, 130),
                                       (64, 3, 8, 18)])
def test_many_rows_match_oracle(d, hkv, g, m, wide):
    """More query columns than the decode form holds: every number of pages in the last tile of
    tokens, with and without a tail behind it, rows at the end, all over, and padded."""
    lens = [5, 16, 16 * 3 + 1, 16 * 6 + 15, 16 * 7 + 4, 16 * 8, 16 * 8 + 2, 16 * 11 + 9, 16 * 15 + 3,
            16 * 20, 1333, 0, 2500]
    b = len(lens)
    s = K.Sequences(b, hkv, hkv * g, d, 2500, seed=m + d)
    s.place(lens)
    q = K8.queries(s.rng, b, m, hkv * g, d)
    pos = np.array([[L - m + i for i in range(m)] for L in lens])
    pos[pos < 0] = -1
    pos[10] = s.rng.integers(0, 1333, m)
    got = s.attend(q, pos, wide=wide)
    assert (got[pos < 0] == 0).all()
    # all the short sequences, and of the long ones every third row
    s.check_attention(got[:10], q[:10], pos[:10], lens=np.array(lens[:10]))
    thin, some = pos.copy(), got.copy()
    keep = np.arange(m) % 3 == 0
    thin[:, ~keep], some[:, ~keep] = -1, 0
    s.check_attention(some, q, thin, heads={(i, h) for i in (10, 11, 12) for h in range(hkv)})
    assert H.status(s.cache) == 0
    pos[0, 0] = 5
    assert (s.attend(q, pos, wide=wide)[0, 0] == 0).all() and H.status(s.cache) == H.lib().DEVERR_SEQ_LEN


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("m", [9, 27])
def test_odd_tails_and_bad_pages(m, wide):
    """NaN and infinities in the tail reach the rows that see them only; refused pages and tails are
    left out, whatever page 0 holds, and reported."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 1, 2, 64, 700)
    k, v = K8.draw(s.rng, 90 + 650, 1, 64)
    v[85, 0, 7], v[86, 0, 9], k[88, 0, 3] = np.nan, np.inf, np.nan
    s.place([90, 650], k, v)
    pos = np.array([[79, 84, 85, 86, 87, 88, 89, 80, -1] * (m // 9), np.arange(650 - m, 650)])
    q = K8.queries(s.rng, 2, m, 2, 64)
    got = s.attend(q, pos, wide=wide)
    for i in range(0, m, 9):
        assert np.isfinite(got[0, [i, i + 1, i + 7, i + 8]]).all()
        assert np.isnan(got[0, i + 2, :, 7]).all() and np.isfinite(np.delete(got[0, i + 2], 7, -1)).all()
        assert np.isinf(got[0, i + 3, :, 9]).all() and np.isnan(got[0, i + 5]).all()
    clean, seen = got.copy(), pos.copy()
    for i in range(m):
        if i % 9 in (2, 3, 4, 5, 6):
            clean[0, i], seen[0, i] = 0, -1
    s.check_attention(clean, q, seen)
    drop = sorted({3, 33} | set(np.flatnonzero(s.table[1] == 0).tolist()))
    s.cache.pool[0].fill_(0xFF)
    for p, bad in zip(drop, (-1, s.cache.pool.shape[0], -7)):
        s.cache.page_table[1, p] = bad
    got = s.attend(q, pos, wide=wide)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    s.check_attention(got, q, pos, drop=drop, heads={(1, 0)})
    s.cache.tail_ids = s.i32([0, -1])
    got = s.attend(q, pos, wide=wide)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    s.check_attention(got, q, pos, drop=drop + [40], heads={(1, 0)})


@pytest.mark.parametrize("hkv,g,n", [(8, 4, 40013), (2, 8, 40013), (8, 8, 20000)])
def test_long_context(hkv, g, n):
    """One sequence over every CTA of the grid."""
    s = K.Sequences(1, hkv, hkv * g, 128, n, seed=3)
    s.place([n])
    q = K8.queries(s.rng, 1, 1, hkv * g, 128)
    s.check_attention(s.attend(q), q, heads={(0, 0), (0, hkv - 1)})


@pytest.mark.parametrize("batch,hkv,d,lo,hi,m", [
    (300, 4, 64, 0, 120, 1), (170, 1, 64, 1, 90, 1), (330, 4, 128, 0, 40, 1), (900, 3, 64, 0, 33, 1),
    (90, 2, 128, 1, 2300, 1), (3, 60, 128, 2000, 2400, 1), (200, 1, 64, 2000, 2200, 1),
    (1, 2, 128, 900, 900, 14), (20, 4, 128, 30, 300, 8), (30, 1, 64, 1500, 3000, 12), (12, 3, 128, 700, 1900, 5),
    (40, 2, 128, 300, 700, 16), (3, 2, 128, 3000, 5000, 31)])
def test_every_split_of_the_work(batch, hkv, d, lo, hi, m):
    """Teams, clusters and equal shares, one tile of columns and several: sampled units."""
    rng = np.random.default_rng(hi)
    lens = rng.integers(lo, hi + 1, batch)
    lens[0], lens[-1] = lo, hi
    s = K.Sequences(batch, hkv, 2 * hkv, d, hi, seed=batch)
    s.place(lens)
    q = K8.queries(s.rng, batch, m, 2 * hkv, d)
    pos = None
    if m > 1:
        pos = np.maximum(lens[:, None] - m + np.arange(m), -1)
        pos[0, -1] = -1                    # a padded row
        pos[-1, 0] = lens[-1] - 1          # and one out of order
    got = s.attend(q, pos)
    heads = {(int(b), int(h)) for b, h in zip(rng.integers(0, batch, 60 // m + 3), rng.integers(0, hkv, 60 // m + 3))}
    s.check_attention(got, q, pos, heads=heads | {(0, 0), (batch - 1, hkv - 1)})
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("m", [1, 3, 6, 40])
def test_scales_of_values_and_queries(m, wide):
    """Value scales that differ by 2^20 from page to page, in both directions; pages, and a tail, of
    zeros among them; queries from 1e-20 to 1e4 (logits to saturation); each form of the kernel."""
    s = K.Sequences(2, 1, 4, 128, 1500, seed=9)
    k, v = K8.draw(s.rng, 1500 + 907, 1, 128)
    grow = np.exp2(np.arange(1500) // 16 % 41 - 20.0)[:, None, None].astype(np.float32)
    v[:1500] *= grow
    v[1500:] /= grow[:907]
    v[320:352] = 0
    v[1500 + 896:] = 0
    s.place([1500, 907], k, v)
    for scale in (1e-20, 1.0, 1e4):
        q = K8.queries(s.rng, 2, m, 4, 128, scale)
        pos = None if m == 1 else np.array([[1500 - m + i for i in range(m)], [907 - m + i for i in range(m)]])
        s.check_attention(s.attend(q, pos, wide=wide), q, pos)
    s.check_pools()


@pytest.mark.parametrize("m", [1, 5, 40])
@pytest.mark.parametrize("scale", [2.0 ** -90, 1e25])
def test_values_far_from_unit_scale(m, scale):
    """Values of any size: the page's scale is outside the fp16 arithmetic."""
    s = K.Sequences(2, 1, 4, 128, 700, seed=m)
    k, v = K8.draw(s.rng, 645 + 151, 1, 128)
    v = synth.bf16_round((v.astype(np.float64) * scale).astype(np.float32))
    s.place([645, 151], k, v)
    q = K8.queries(s.rng, 2, m, 4, 128)
    pos = None if m == 1 else np.array([np.arange(x - m, x) for x in (645, 151)])
    s.check_attention(s.attend(q, pos), q, pos)


def test_bad_lengths_are_reported():
    L = H.lib()
    s = K.Sequences(2, 2, 4, 128, 400)
    s.place([390, 100])
    q = K8.queries(s.rng, 2, 1, 4, 128)
    good = s.attend(q)
    got = s.attend(q, lens=[-3, 401], max_len=400)
    assert H.status(s.cache) == L.DEVERR_SEQ_LEN and (got == 0).all()
    s.cache.status.zero_()
    np.testing.assert_array_equal(s.attend(q), good)
    assert H.status(s.cache) == 0


def test_page_offsets_beyond_4_gib():
    """Page ids whose blocks lie past 2^32 bytes."""
    t = H.torch()
    s = K.Sequences(1, 8, 8, 128, 64)
    need = (5 << 30) // (8 * 2320)
    s.cache.pool = t.empty((need, 8, 2320), dtype=t.uint8, device=H.DEV)
    ids = np.array([need - 1, 3, need - 2, need // 2 + 1], np.int32)
    s.cache.page_table.copy_(t.from_numpy(ids[None]))
    s.place([64])
    q = K8.queries(s.rng, 1, 1, 8, 128)
    s.check_attention(s.attend(q), q)
    rows, pos = K8.queries(s.rng, 1, 20, 8, 128), np.arange(44, 64)[None]
    for wide in WIDE:
        s.check_attention(s.attend(rows, pos, wide=wide), rows, pos)
    k, v = (t.empty((64, 8, 128), dtype=t.bfloat16, device=H.DEV) for _ in range(2))
    H.lib().oscar_kv4_gather(s.cache, s.i32([64]), s.i32([0]), s.i32([0, 64]), 64, k, v)
    for h in range(8):
        for got, want in zip((k, v), s.stored(0, h)):
            np.testing.assert_array_equal(H.from_bf16(got)[:, h], synth.bf16_round(want.astype(np.float32)))
    blk = s.cache.pool[int(ids[0]), 7].cpu().numpy()
    np.testing.assert_array_equal(blk, kv4.block_bytes(s.k[0][:16, 7], s.v[0][:16, 7]))


@pytest.mark.parametrize("m,n", [(1, 3000), (5, 3000), (65, 3000), (1, 200)])
def test_same_bits_again_on_two_streams_and_from_graphs(m, n):
    """The same call with dirty workspaces, two streams at once with a workspace each, and two
    captured calls with theirs, replayed after their inputs changed."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(3, 4, 16, 128, n + 200, seed=2)
    s.place([n, 77, n // 2])
    q = K8.queries(s.rng, 3, m, 16, 128)

    def positions():
        return None if m == 1 else np.maximum(s.lens[:, None] - m + np.arange(m), -1)

    pos, top = positions(), n + 200
    want = s.attend(q, pos, max_len=top)
    some = {(0, 1), (1, 3), (2, 0)}
    s.check_attention(want, q, pos, heads=some)
    np.testing.assert_array_equal(want, s.attend(q, pos, max_len=top))
    qt, lens = H.bf16_tensor(q if m > 1 else q[:, 0]), s.i32(s.lens)
    at = None if m == 1 else s.i32(pos)
    size = L.oscar_kv4_workspace_size(s.cache, 3, m, top)
    outs = [t.zeros_like(qt) for _ in range(6)]
    spaces = [t.full((size,), 0x7F, dtype=t.uint8, device=H.DEV) for _ in range(2)]
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    for i in range(6):
        L.oscar_kv4_attention(s.cache, qt, lens, top, outs[i], spaces[i % 2], q_pos=at, stream=streams[i % 2])
    t.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(H.from_bf16(o).reshape(want.shape), want)
    graphs = [t.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with t.cuda.graph(graph):
            L.oscar_kv4_attention(s.cache, qt, lens, top, outs[i], spaces[i], q_pos=at)
        outs[i].zero_()
    for graph in graphs:
        graph.replay()
    t.cuda.synchronize()
    for o in outs[:2]:
        np.testing.assert_array_equal(H.from_bf16(o).reshape(want.shape), want)
    s.place([40, 3, 1])
    q = K8.queries(s.rng, 3, m, 16, 128)
    lens.copy_(s.i32(s.lens)), qt.copy_(H.bf16_tensor(q if m > 1 else q[:, 0]))
    if m > 1:
        at.copy_(s.i32(positions()))
    for graph in graphs * 2:
        graph.replay()
    t.cuda.synchronize()
    for o in outs[:2]:
        s.check_attention(H.from_bf16(o).reshape(want.shape), q, positions(), heads=some)


def test_a_serving_loop():
    """Prompts admitted, then chunks and single tokens: pages from a free list, rotary positions,
    placing, attention of the new rows, and the prefix read back, all from the same lists."""
    t, L = H.torch(), H.lib()
    b, hkv, g, d, maxp = 3, 2, 4, 128, 24
    rng = np.random.default_rng(11)
    cache = pages.allocate_kv4(b * maxp, b, maxp, hkv=hkv, hq=hkv * g, d=d, device=H.DEV)
    i32 = dict(dtype=t.int32, device=H.DEV)
    free = t.from_numpy(rng.permutation(b * maxp).astype(np.int32)).to(H.DEV)
    lens, cursor = t.zeros(b, **i32), t.zeros(1, **i32)
    freq = 1e6 ** (-2.0 * np.arange(d // 2) / d) / (2 * np.pi)
    phases = t.from_numpy(L.oscar_rope_phases(1e6, d).view(np.int64)).to(H.DEV)
    raw_k = [np.zeros((0, hkv, d)) for _ in range(b)]
    raw_v = [np.zeros((0, hkv, d), np.float32) for _ in range(b)]
    n_lens = np.zeros(b, int)
    for new in ([200, 37, 16], [1, 1, 1], [16, 0, 9], [1, 1, 1]):
        n, m = sum(new), max(new)
        before = lens.clone()
        ps, rs = t.empty(b + 1, **i32), t.empty(b + 1, **i32)
        ids, pos = t.empty(n, **i32), t.empty(n, **i32)
        L.oscar_extend_pages(cache.page_table, lens, t.tensor(new, **i32), free, cursor, lens, ps, rs, ids, pos,
                             hold_back=15, status=cache.status)
        cursor = ps[-1:].clone()
        k, v = K8.draw(rng, n, hkv, d)
        q = K8.queries(rng, n, 1, hkv * g, d)[:, 0]
        kt, qt = H.bf16_tensor(k), H.bf16_tensor(q)
        L.oscar_rope(qt, kt, pos, phases)
        L.oscar_kv4_place(cache, kt, H.bf16_tensor(v), before, rs, m)
        # queries as [b][m], rows of sequences that bring fewer are padded
        rows = t.zeros(b, m, hkv * g, d, dtype=t.bfloat16, device=H.DEV)
        q_pos = t.full((b, m), -1, **i32)
        at = pos - before[ids.long()]
        rows[ids.long(), at.long()] = qt
        q_pos[ids.long(), at.long()] = pos
        out = t.full_like(rows, float("nan"))
        top = int(lens.max())
        ws = t.empty(L.oscar_kv4_workspace_size(cache, b, m, top), dtype=t.uint8, device=H.DEV)
        L.oscar_kv4_attention(cache, rows, lens, top, out, ws, q_pos=q_pos)
        t.cuda.synchronize()
        assert H.status(cache) == 0
        kr, at0 = H.from_bf16(kt), 0
        got, qr = H.from_bf16(out), H.from_bf16(rows)
        want_k = kv8.rope(k.astype(np.float64), pos.cpu().numpy(), freq, False)
        assert np.abs(kr - want_k).max() <= 2.0 ** -7 * np.abs(want_k).max()   # two bf16 steps of the largest
        for i in range(b):
            raw_k[i] = np.concatenate([raw_k[i], kr[at0:at0 + new[i]]])
            raw_v[i] = np.concatenate([raw_v[i], v[at0:at0 + new[i]]])
            at0 += new[i]
            first = n_lens[i]
            n_lens[i] += new[i]
            for h in range(hkv):
                sk, sv = kv4.stored(raw_k[i][:, h], False), kv4.stored(raw_v[i][:, h], True)
                for r in range(m):
                    for j in range(g):
                        limit = first + r + 1 if r < new[i] else 0
                        ref, w = kv8.attention(qr[i, r, h * g + j], sk, sv, limit)
                        # as kv8_harness.check_attention: logits 2^-17 (unit-scale keys, 128 products),
                        # weights 2^-12, sums 2^-18, output 2^-8
                        e = 2 * 24 * 2.0 ** -23 * np.abs(qr[i, r, h * g + j]).sum() * np.abs(sk).max() / np.sqrt(d)
                        e += 2.0 ** -20 * (np.abs(sk[:limit] @ qr[i, r, h * g + j]).max() if limit else 0)
                        tol = (2.0 ** -12 + e + 2.0 ** -17) * w + 2.0 ** -30 * limit * np.abs(sv).max()
                        tol += 2.0 ** -8 * (np.abs(ref) + tol)
                        assert (np.abs(got[i, r, h * g + j] - ref) <= tol).all()
    starts = t.tensor(np.concatenate([[0], np.cumsum(n_lens)]), **i32)
    ko, vo = (t.empty((int(n_lens.sum()), hkv, d), dtype=t.bfloat16, device=H.DEV) for _ in range(2))
    L.oscar_kv4_gather(cache, lens, t.zeros(b, **i32), starts, int(n_lens.max()), ko, vo)
    ko, vo, at0 = H.from_bf16(ko), H.from_bf16(vo), 0
    for i in range(b):
        for h in range(hkv):
            for got, x, value in ((ko, raw_k, False), (vo, raw_v, True)):
                want = synth.bf16_round(kv4.stored(x[i][:, h], value).astype(np.float32))
                np.testing.assert_array_equal(got[at0:at0 + n_lens[i], h], want)
        at0 += n_lens[i]
    assert H.status(cache) == 0


def test_binding_refuses_tensors():
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 2, 4, 64, 100)
    s.place([20, 30])
    k = t.zeros(3, 2, 64, dtype=t.bfloat16, device=H.DEV)
    i = s.i32([0, 1, 3])
    for bad in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=k.cpu()), dict(lens=i), dict(lens=i[:2].long()),
                dict(starts=i[:2])):
        a = dict(dict(k=k, v=k, lens=i[:2], starts=i), **bad)
        with pytest.raises(ValueError):
            L.oscar_kv4_place(s.cache, a["k"], a["v"], a["lens"], a["starts"], 3)
    with pytest.raises(ValueError):
        L.oscar_kv4_place(s.cache, k, k, i[:2], i, 1 << 31)
    q = t.zeros(2, 4, 64, dtype=t.bfloat16, device=H.DEV)
    ws = t.empty(1 << 20, dtype=t.uint8, device=H.DEV)
    for args in ((q[:, :2], i[:2], 30, q), (q, i[:2], 30, q.float()), (q, i[:2].cpu(), 30, q)):
        with pytest.raises(ValueError):
            L.oscar_kv4_attention(s.cache, *args, ws)
    with pytest.raises(ValueError):
        L.oscar_kv4_gather(s.cache, i[:2], i[:2], i, 3, k[:, :, :32], k)
    with pytest.raises(L.OscarError):
        L.oscar_kv4_attention(s.cache, q, i[:2], 0, q, ws)


@pytest.mark.parametrize("most", [(1 << 31) - 1, (1 << 31) - 20])
def test_a_bound_of_rows_that_says_nothing(most):
    """max_new and max_rows of all that an int32 holds: the rows that there are bound the work."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(1, 3, 3, 64, 400, seed=4)
    s.place([21], max_new=most)
    s.place([302], max_new=most)
    s.check_pools()
    k, v = (t.full((325, 3, 64), 7.0, dtype=t.bfloat16, device=H.DEV) for _ in range(2))
    L.oscar_kv4_gather(s.cache, s.i32([323]), s.i32([5]), s.i32([0, 318]), most, k, v)
    for h in range(3):
        for got, want in zip((k, v), s.stored(0, h)):
            np.testing.assert_array_equal(H.from_bf16(got)[:318, h], synth.bf16_round(want[5:].astype(np.float32)))
    assert (k[318:] == 7).all() and (v[318:] == 7).all()
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("m,top", [(1, 4100), (3, 4100), (5, 4100), (5, 40000)])
def test_short_and_empty_sequences_among_long_ones(m, top):
    """Shares that end before a unit's pages, in them and behind them; sequences without a token."""
    lens = np.array([3000, 0, 1, 5, 16, 0, 0, 700, 17, 40, 2, 0, 1500, 31, 0] * 2)
    s = K.Sequences(len(lens), 8, 32, 128, 4096, seed=m)
    s.place(lens)
    q = K8.queries(s.rng, len(lens), m, 32, 128)
    pos = None if m == 1 else np.maximum(s.lens[:, None] - m + np.arange(m), -1)
    got = s.attend(q, pos, wide=top // 16)
    some = {(b, h) for b in range(len(lens)) for h in ((b % 8, 7 - b % 8) if lens[b] > 1000 else range(8))}
    s.check_attention(got, q, pos, heads=some)
    assert H.status(s.cache) == 0
    np.testing.assert_array_equal(got, s.attend(q, pos, wide=top // 16))

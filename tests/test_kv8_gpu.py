"""GPU parity of the 8-bit cache: placement byte for byte, reading back, attention of
one and several rows, against the fp64 oracle; and what the calls refuse or report."""
import numpy as np
import pytest

import gpu_harness as H
import kv8_harness as K
from int2_rotated_kv_gb300 import synth
from oracle import kv8

pytestmark = pytest.mark.gpu

FMTS = [kv8.INT8, kv8.E4M3]
WIDE = [0, 131072]   # see kv8_harness.Sequences.attend


# ---------------------------------------------------------------------- placing

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3), (128, 8), (64, 5)])
def test_placing_in_any_pieces_gives_the_same_pages(fmt, d, hkv):
    """Prompts, chunks that start and end inside pages, single tokens, sequences that
    rest: pages and tails byte for byte after every call."""
    s = K.Sequences(5, hkv, hkv, d, fmt, 140, seed=d + hkv + fmt, permute_tails=hkv == 3)
    for new in ([1, 0, 15, 16, 17], [1, 5, 1, 1, 31], [16, 11, 0, 47, 1], [13, 1, 33, 2, 0],
                [1, 1, 1, 1, 1], [20, 0, 15, 3, 40]):
        s.place(new, packed=hkv == 8)
        s.check_pools()
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_placing_special_values(fmt):
    """Zero and tiny blocks, the largest and smallest bf16 values, NaN and infinities."""
    d, hkv = 64, 1
    s = K.Sequences(1, hkv, hkv, d, fmt, 200)
    k, v = K.draw(s.rng, 16 * 9 + 5, hkv, d)
    big = float(synth.bf16_from_bits(np.array([0x7F7F], np.uint16))[0])
    k[0:16] = 0.0
    k[16:32] = synth.bf16_round(np.full((16, 1, d), 2.0 ** -101, np.float32))
    k[32:48] = 2.0 ** -100
    k[48] = big
    v[48:64] *= np.float32(2.0 ** -90)
    v[0, 0, 0] = -big
    k[64, 0, 3], k[65, 0, 4], k[66, 0, 5] = np.nan, np.inf, -np.inf
    v[80:96] = np.nan
    v[96:112] = np.inf
    v[97, 0, 1] = -1e-39          # a subnormal, and nothing else that is finite
    k[112:128, 0] = np.linspace(-1, 1, 16 * d).reshape(16, d)
    k[112:128] = synth.bf16_round(k[112:128])
    k[148, 0, 0] = np.nan         # stays in the tail as it is
    s.place([16 * 9 + 5], k, v)
    s.check_pools()
    assert H.status(s.cache) == H.lib().DEVERR_NONFINITE


def test_rows_behind_the_last_sequence_and_other_streams():
    """Rows that belong to no sequence are not read; a call on another stream."""
    t = H.torch()
    s = K.Sequences(3, 2, 2, 128, kv8.INT8, 100)
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(stream):
        s.place([33, 0, 20], extra_rows=7)
    s.place([1, 2, 0], stream=stream, max_new=50)
    stream.synchronize()
    s.check_pools()


def test_placing_reports_what_it_skips():
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 1, 1, 64, kv8.INT8, 64)
    s.place([10, 20])
    k, v = (H.bf16_tensor(x) for x in K.draw(s.rng, 30, 1, 64))

    def call(lens, starts, max_new):
        L.oscar_kv8_place(s.cache, k, v, s.i32(lens), s.i32(starts), max_new)
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


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv", [(64, 2), (128, 3)])
def test_gather(fmt, d, hkv):
    t, L = H.torch(), H.lib()
    s = K.Sequences(4, hkv, hkv, d, fmt, 120, seed=7)
    s.place([100, 0, 31, 64])
    first, count = np.array([3, 0, 30, 16]), np.array([97, 0, 1, 33])
    starts = np.concatenate([[0], np.cumsum(count)])
    n = starts[-1]
    ko, vo = (t.full((n + 2, hkv, d), 7.0, dtype=t.bfloat16, device=H.DEV) for _ in range(2))
    L.oscar_kv8_gather(s.cache, s.i32(s.lens), s.i32(first), s.i32(starts), 97, ko, vo)
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
    L.oscar_kv8_gather(s.cache, s.i32(s.lens), s.i32([4, 0, 0, 0]), s.i32(starts), 97, ko, vo)
    assert H.status(s.cache) == L.DEVERR_SEQ_LEN                      # 4 + 97 > 100 tokens
    assert (ko[:97] == 7).all()


# -------------------------------------------------------------------- attention

@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv,g", [(64, 1, 4), (128, 2, 1), (128, 2, 4), (64, 3, 3), (128, 1, 8),
                                     (128, 1, 16), (64, 1, 40)])
def test_decode_matches_oracle(fmt, d, hkv, g, wide):
    """Ragged lengths, with none, one token, and ends on and beside page borders."""
    lens = [0, 1, 15, 16, 17, 33, 700, 2607, 1024]
    s = K.Sequences(len(lens), hkv, hkv * g, d, fmt, 2700, seed=g)
    s.place(lens)
    q = K.queries(s.rng, len(lens), 1, hkv * g, d)
    got = s.attend(q, wide=wide)
    s.check_attention(got, q)
    assert H.status(s.cache) == 0
    # fewer tokens than placed pages hold: whole pages are read from the pool all the same
    short = np.array([0, 1, 15, 16, 16, 32, 688, 1600, 1008])
    s2 = s.attend(q, lens=short, wide=wide)
    for b in (4, 5, 6, 7, 8):
        one = np.zeros_like(short)
        one[b] = short[b]
        s.check_attention(s2, q, lens=one, heads={(b, h) for h in range(hkv)})


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv,g,m", [(64, 1, 4, 2), (128, 2, 4, 3), (128, 1, 1, 11), (128, 2, 4, 9),
                                       (64, 2, 8, 5), (128, 1, 3, 37)])
def test_rows_match_oracle(fmt, d, hkv, g, m, wide):
    """Several rows: the last positions, positions all over the context in no order,
    rows that see nothing, and rows behind the end (zeros, reported)."""
    lens = [40, 0, 555, 1700]
    s = K.Sequences(4, hkv, hkv * g, d, fmt, 1800, seed=m)
    s.place(lens)
    q = K.queries(s.rng, 4, m, hkv * g, d)
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
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hkv,g,m", [(128, 2, 1, 17), (64, 1, 2, 64), (128, 1, 4, 33), (128, 1, 2, 130),
                                       (64, 3, 8, 18)])
def test_many_rows_match_oracle(fmt, d, hkv, g, m, wide):
    """More query columns than the decode form holds, one tile of 128 and several: every
    number of pages in the last tile of tokens, with and without a tail behind it, rows at
    the end, all over, and padded."""
    lens = [5, 16, 16 * 3 + 1, 16 * 6 + 15, 16 * 7 + 4, 16 * 8, 16 * 8 + 2, 16 * 11 + 9, 16 * 15 + 3,
            16 * 20, 1333, 0, 2500]
    b = len(lens)
    s = K.Sequences(b, hkv, hkv * g, d, fmt, 2500, seed=m + d)
    s.place(lens)
    q = K.queries(s.rng, b, m, hkv * g, d)
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
def test_many_rows_with_odd_tails_and_bad_pages(wide):
    """NaN and infinities in the tail reach the rows that see them only; refused pages and
    tails are left out and reported."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 1, 2, 64, kv8.INT8, 700)
    k, v = K.draw(s.rng, 90 + 650, 1, 64)
    v[85, 0, 7], v[86, 0, 9], k[88, 0, 3] = np.nan, np.inf, np.nan
    s.place([90, 650], k, v)
    pos = np.array([[79, 84, 85, 86, 87, 88, 89, 80, -1] * 3, np.arange(650 - 27, 650)])
    q = K.queries(s.rng, 2, 27, 2, 64)
    got = s.attend(q, pos, wide=wide)
    for i in (0, 9, 18):
        assert np.isfinite(got[0, [i, i + 1, i + 7, i + 8]]).all()
        assert np.isnan(got[0, i + 2, :, 7]).all() and np.isfinite(np.delete(got[0, i + 2], 7, -1)).all()
        assert np.isinf(got[0, i + 3, :, 9]).all() and np.isnan(got[0, i + 5]).all()
    clean, seen = got.copy(), pos.copy()
    for i in range(27):
        if i % 9 in (2, 3, 4, 5, 6):
            clean[0, i], seen[0, i] = 0, -1
    s.check_attention(clean, q, seen)
    s.cache.page_table[1, 3] = -1
    s.cache.page_table[1, 33] = s.cache.pool.shape[0]
    got = s.attend(q, pos, wide=wide)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    s.check_attention(got, q, pos, drop=(3, 33), heads={(1, 0)})
    s.cache.page_table.copy_(t.from_numpy(s.table))
    s.cache.status.zero_()
    s.cache.tail_ids = s.i32([0, -1])
    got = s.attend(q, pos, wide=wide)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    s.check_attention(got, q, pos, drop=(40,), heads={(1, 0)})


@pytest.mark.parametrize("fmt,hkv,g", [(kv8.INT8, 8, 4), (kv8.E4M3, 2, 8)])
def test_long_context(fmt, hkv, g):
    """One sequence over every CTA of the grid."""
    n = 40013
    s = K.Sequences(1, hkv, hkv * g, 128, fmt, n, seed=3)
    s.place([n])
    q = K.queries(s.rng, 1, 1, hkv * g, 128)
    got = s.attend(q)
    s.check_attention(got, q, heads={(0, 0), (0, hkv - 1)})


def test_many_short_sequences():
    """More units than CTAs: several units per CTA, units over CTA borders."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 120, 300)
    s = K.Sequences(300, 4, 8, 64, kv8.INT8, 120, seed=5)
    s.place(lens)
    q = K.queries(s.rng, 300, 1, 8, 64)
    got = s.attend(q, max_len=120)
    s.check_attention(got, q)
    got2 = s.attend(q, max_len=120 + 7)          # another max_len: other shares, no other results
    s.check_attention(got2, q)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch,hkv,d,lo,hi", [
    (170, 1, 64, 1, 90), (330, 2, 64, 0, 60), (330, 4, 128, 0, 40), (900, 3, 64, 0, 33),
    (90, 2, 128, 1, 2300), (3, 60, 128, 2000, 2400), (200, 1, 64, 2000, 2200)])
def test_every_split_of_the_work(fmt, batch, hkv, d, lo, hi):
    """Teams of 8, 4, 2 and 1 warps, and equal shares over many units: sampled units."""
    rng = np.random.default_rng(hi)
    lens = rng.integers(lo, hi + 1, batch)
    lens[0], lens[-1] = lo, hi
    s = K.Sequences(batch, hkv, 2 * hkv, d, fmt, hi, seed=batch)
    s.place(lens)
    q = K.queries(s.rng, batch, 1, 2 * hkv, d)
    got = s.attend(q)
    heads = {(int(b), int(h)) for b, h in zip(rng.integers(0, batch, 60), rng.integers(0, hkv, 60))}
    s.check_attention(got, q, heads=heads | {(0, 0), (batch - 1, hkv - 1)})
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 6])
def test_scales_of_values_and_queries(fmt, m, wide):
    """Value scales that differ by 2^20 from page to page, in both directions; queries from
    1e-20 to 1e4 (logits to saturation); each form of the kernel."""
    s = K.Sequences(2, 1, 4, 128, fmt, 1500, seed=9)
    k, v = K.draw(s.rng, 1500 + 900, 1, 128)
    grow = np.exp2(np.arange(1500) // 16 % 41 - 20.0)[:, None, None].astype(np.float32)
    v[:1500] *= grow
    v[1500:] /= grow[:900]
    s.place([1500, 900], k, v)
    for scale in (1e-20, 1.0, 1e4):
        q = K.queries(s.rng, 2, m, 4, 128, scale)
        pos = None if m == 1 else np.array([[1500 - m + i for i in range(m)], [900 - m + i for i in range(m)]])
        s.check_attention(s.attend(q, pos, wide=wide), q, pos)
    s.check_pools()


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
def test_pages_of_zeros_among_small_values(fmt, m, wide):
    """Values of 1e-5 beside pages, and a tail, whose values are all zero: the zeros' weights
    count, and take no precision from the others."""
    s = K.Sequences(3, 1, 4, 128, fmt, 700, seed=m)
    n = np.array([650, 16 * 20, 16 * 9 + 7])
    k, v = K.draw(s.rng, int(n.sum()), 1, 128)
    v = synth.bf16_round(v * np.float32(1e-5))
    v[32:64] = 0
    v[16 * 30:16 * 31] = 0
    v[640:650] = 0                    # the first sequence's tail
    v[650:650 + 16 * 19] = 0          # all but the second's last page
    s.place(n, k, v)
    q = K.queries(s.rng, 3, m, 4, 128)
    pos = None if m == 1 else np.stack([np.arange(x - m, x) for x in n])
    s.check_attention(s.attend(q, pos, wide=wide), q, pos)
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
def test_a_token_that_a_row_does_not_see_does_not_reach_it(wide):
    """NaN and infinity in the tail: rows before them keep finite outputs, rows behind
    them get what the softmax gives."""
    s = K.Sequences(1, 1, 2, 64, kv8.INT8, 100)
    k, v = K.draw(s.rng, 90, 1, 64)
    v[85, 0, 7], v[86, 0, 9], k[88, 0, 3] = np.nan, np.inf, np.nan
    s.place([90], k, v)
    pos = np.array([[79, 84, 85, 86, 87, 88, 89, 80, -1]])
    q = K.queries(s.rng, 1, 9, 2, 64)
    got = s.attend(q, pos, wide=wide)
    assert np.isfinite(got[0, [0, 1, 7, 8]]).all()
    assert np.isnan(got[0, 2, :, 7]).all() and np.isfinite(np.delete(got[0, 2], 7, -1)).all()
    assert np.isinf(got[0, 3, :, 9]).all() and np.isnan(got[0, 5]).all()
    finite = np.array([[79, 84, -1, -1, -1, -1, -1, 80, -1]])
    clean = got.copy()
    clean[0, 2:7] = 0
    s.check_attention(clean, q, finite)


def test_queries_that_are_not_finite():
    s = K.Sequences(2, 1, 4, 64, kv8.INT8, 100)
    s.place([70, 50])
    q = K.queries(s.rng, 2, 1, 4, 64)
    q[0, 0, 1, 5] = np.nan
    q[0, 0, 2] = 0.0
    got = s.attend(q)
    assert np.isnan(got[0, 0, 1]).all()
    rest = got.copy()
    q[0, 0, 1, 5] = 0.0
    rest[0, 0, 1] = s.attend(q)[0, 0, 1]
    s.check_attention(rest, q)


def test_bad_pages_and_lengths_are_reported_and_left_out():
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 2, 4, 128, kv8.E4M3, 400)
    s.place([390, 100])
    q = K.queries(s.rng, 2, 1, 4, 128)
    good = s.attend(q)
    s.cache.page_table[0, 3] = -1
    s.cache.page_table[0, 9] = s.cache.pool.shape[0]
    got = s.attend(q)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    s.check_attention(got, q, drop=(3, 9), heads={(0, 0), (0, 1)})
    np.testing.assert_array_equal(got[1], good[1])
    s.cache.page_table.copy_(t.from_numpy(s.table))
    s.cache.status.zero_()
    s.cache.tail_ids = s.i32([s.cache.tail.shape[0], 1])
    got = s.attend(q)
    assert H.status(s.cache) == L.DEVERR_PAGE_ID
    s.check_attention(got, q, drop=(24,), heads={(0, 0), (0, 1)})
    s.cache.tail_ids = None
    s.cache.status.zero_()
    got = s.attend(q, lens=[-3, 401], max_len=400)
    assert H.status(s.cache) == L.DEVERR_SEQ_LEN and (got == 0).all()
    s.cache.status.zero_()
    np.testing.assert_array_equal(s.attend(q), good)


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("m", [1, 3, 200])
def test_a_refused_page_is_left_out_whatever_page_0_holds(m, wide):
    """Codes and scales of all ones (NaN in e4m3 and in fp32) in page 0, ids out of range."""
    s = K.Sequences(1, 2, 8, 128, kv8.E4M3, 800, seed=7)
    s.place([733])
    drop = sorted({3, 40} | set(np.flatnonzero(s.table[0] == 0).tolist()))
    s.cache.pool[0].fill_(0xFF)
    table = s.table.copy()
    table[0, drop] = [-1, len(s.ids), -7][:len(drop)]
    s.cache.page_table.copy_(H.torch().from_numpy(table))
    s.cache.status = s.i32([0])
    q = K.queries(s.rng, 1, m, 8, 128)
    pos = None if m == 1 else np.arange(733 - m, 733)[None]
    s.check_attention(s.attend(q, pos, wide=wide), q, pos, drop=drop)
    assert H.status(s.cache) == H.lib().DEVERR_PAGE_ID


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b,m,d,hkv,g,lo,hi", [
    (1, 7, 128, 2, 4, 900, 900),       # clusters, several tiles of 8 columns
    (3, 5, 64, 2, 8, 100, 400),
    (1, 50, 128, 2, 4, 500, 500),      # teams
    (20, 4, 128, 4, 4, 30, 300),
    (30, 6, 64, 1, 4, 1500, 3000),     # shares
])
def test_several_tiles_of_eight_columns(fmt, b, m, d, hkv, g, lo, hi, wide):
    """Rows that fill several narrow tiles, the last one partly, in each division of the work."""
    s = K.Sequences(b, hkv, hkv * g, d, fmt, hi, seed=b + m)
    n = s.rng.integers(lo, hi + 1, b)
    s.place(n)
    q = K.queries(s.rng, b, m, hkv * g, d)
    pos = np.maximum(n[:, None] - m + np.arange(m), -1)
    pos[0, -1] = -1                    # a padded row
    pos[-1, 0] = n[-1] - 1             # and one out of order
    got = s.attend(q, pos, wide=wide)
    s.check_attention(got, q, pos)
    assert not got[0, -1].any() and H.status(s.cache) == 0


def test_page_offsets_beyond_4_gib():
    """Page ids whose blocks lie past 2^32 bytes."""
    t = H.torch()
    s = K.Sequences(1, 8, 8, 128, kv8.INT8, 64)
    need = (5 << 30) // (8 * 4112)
    s.cache.pool = t.empty((need, 8, 4112), dtype=t.uint8, device=H.DEV)
    ids = np.array([need - 1, 3, need - 2, need // 2 + 1], np.int32)
    s.cache.page_table.copy_(t.from_numpy(ids[None]))
    s.place([64])
    q = K.queries(s.rng, 1, 1, 8, 128)
    s.check_attention(s.attend(q), q)
    rows, pos = K.queries(s.rng, 1, 20, 8, 128), np.arange(44, 64)[None]
    for wide in WIDE:
        s.check_attention(s.attend(rows, pos, wide=wide), rows, pos)
    k, v = (t.empty((64, 8, 128), dtype=t.bfloat16, device=H.DEV) for _ in range(2))
    H.lib().oscar_kv8_gather(s.cache, s.i32([64]), s.i32([0]), s.i32([0, 64]), 64, k, v)
    for h in range(8):
        for got, want in zip((k, v), s.stored(0, h)):
            np.testing.assert_array_equal(H.from_bf16(got)[:, h], synth.bf16_round(want.astype(np.float32)))
    order = kv8.orders(128)
    for p, i in enumerate(ids):
        scale, codes = kv8.block(s.v[0][16 * p:16 * p + 16, 7], kv8.INT8)
        blk = s.cache.pool[int(i), 7].cpu().numpy()
        np.testing.assert_array_equal(blk[2048:4096][order[1]], codes)


def test_same_bits_again_and_from_a_graph():
    """The same call twice, with a dirty workspace between, and a captured call replayed
    after its inputs changed: bit-equal outputs."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(3, 4, 16, 128, kv8.INT8, 3100, seed=2)
    s.place([3000, 77, 1500])
    q = K.queries(s.rng, 3, 1, 16, 128)
    a = s.attend(q)
    np.testing.assert_array_equal(a, s.attend(q))
    lens, qt = s.i32(s.lens), H.bf16_tensor(q[:, 0])
    out = t.zeros_like(qt)
    ws = t.full((L.oscar_kv8_workspace_size(s.cache, 3, 1, 3100),), 0x7F, dtype=t.uint8, device=H.DEV)
    stream = t.cuda.Stream()
    with t.cuda.stream(stream):
        L.oscar_kv8_attention(s.cache, qt, lens, 3100, out, ws)
    stream.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        L.oscar_kv8_attention(s.cache, qt, lens, 3100, out, ws)
    out.zero_()
    graph.replay()
    t.cuda.synchronize()
    np.testing.assert_array_equal(H.from_bf16(out), s.attend(q, max_len=3100)[:, 0])
    s.place([40, 3, 1])
    lens.copy_(s.i32(s.lens))
    q2 = K.queries(s.rng, 3, 1, 16, 128)
    qt.copy_(H.bf16_tensor(q2[:, 0]))
    graph.replay()
    graph.replay()
    t.cuda.synchronize()
    s.check_attention(H.from_bf16(out)[:, None], q2)


def test_calls_on_two_streams_with_their_own_workspaces():
    t, L = H.torch(), H.lib()
    s = K.Sequences(2, 8, 32, 128, kv8.E4M3, 5000, seed=4)
    s.place([4999, 2500])
    q = K.queries(s.rng, 2, 1, 32, 128)
    want = s.attend(q)
    qt, lens = H.bf16_tensor(q[:, 0]), s.i32(s.lens)
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in range(2)]
    size = L.oscar_kv8_workspace_size(s.cache, 2, 1, 4999)
    outs = [t.zeros_like(qt) for _ in range(8)]
    spaces = [t.empty(size, dtype=t.uint8, device=H.DEV) for _ in range(2)]
    t.cuda.synchronize()
    for i in range(8):
        L.oscar_kv8_attention(s.cache, qt, lens, 4999, outs[i], spaces[i % 2], stream=streams[i % 2])
    t.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(H.from_bf16(o), want[:, 0])


def test_wide_tiles_on_two_streams_and_from_a_graph():
    """Tiles of 128 columns: the same bits from two streams at once and from a graph, and a
    replay after lengths, positions and queries changed."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(4, 8, 32, 128, kv8.INT8, 3100, seed=9)
    s.place([3000, 1111, 2048, 17])
    q = K.queries(s.rng, 4, 65, 32, 128)
    pos = np.maximum(s.lens[:, None] - 65 + np.arange(65), -1)
    size = L.oscar_kv8_workspace_size(s.cache, 4, 65, 3100)
    assert size > 5 << 20
    want = s.attend(q, pos, max_len=3100)
    some = {(0, 1), (1, 7), (2, 0), (3, 5)}
    s.check_attention(want, q, pos, heads=some)
    qt, lens, at = H.bf16_tensor(q), s.i32(s.lens), s.i32(pos)
    streams = [t.cuda.Stream() for _ in range(2)]
    outs = [t.zeros_like(qt) for _ in range(6)]
    spaces = [t.empty(size, dtype=t.uint8, device=H.DEV) for _ in range(2)]
    t.cuda.synchronize()
    for i in range(6):
        L.oscar_kv8_attention(s.cache, qt, lens, 3100, outs[i], spaces[i % 2], q_pos=at,
                              stream=streams[i % 2])
    t.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(H.from_bf16(o), want)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        L.oscar_kv8_attention(s.cache, qt, lens, 3100, outs[0], spaces[0], q_pos=at)
    outs[0].zero_()
    graph.replay()
    t.cuda.synchronize()
    np.testing.assert_array_equal(H.from_bf16(outs[0]), want)
    s.place([0, 40, 1, 800])
    q = K.queries(s.rng, 4, 65, 32, 128)
    pos = np.maximum(s.lens[:, None] - 65 + np.arange(65), -1)[:, ::-1].copy()
    pos[2, 3:40] = -1
    lens.copy_(s.i32(s.lens)), at.copy_(s.i32(pos)), qt.copy_(H.bf16_tensor(q))
    graph.replay()
    graph.replay()
    t.cuda.synchronize()
    s.check_attention(H.from_bf16(outs[0]), q, pos, heads=some)
    assert H.status(s.cache) == 0


def test_a_descriptor_is_checked_again_when_a_tensor_is_replaced():
    """Also by one at the same address."""
    t, L = H.torch(), H.lib()
    s = K.Sequences(3, 1, 1, 64, kv8.INT8, 100, permute_tails=True)
    s.place([20, 30, 40])
    q = K.queries(s.rng, 3, 1, 1, 64)
    s.attend(q)
    table, tails, pool = s.cache.page_table, s.cache.tail_ids, s.cache.pool
    for name, bad in (("page_table", table.view(t.float32)), ("tail_ids", tails[:2]),
                      ("pool", pool.view(t.int8)), ("tail", s.cache.tail.view(t.float16))):
        good = getattr(s.cache, name)
        setattr(s.cache, name, bad)
        with pytest.raises(ValueError):
            s.attend(q)
        setattr(s.cache, name, good)
    s.check_attention(s.attend(q), q)


FIRST_CALLS = """
import sys
sys.path.insert(0, "tests")
import torch
import kv8_harness as K
from oracle import kv8
from int2_rotated_kv_gb300 import _lib as L
s = K.Sequences(2, 2, 8, 128, kv8.INT8, 400)
new, ws = [300, 77], torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
k, v = K.draw(s.rng, 377, 2, 128)
q = K.queries(s.rng, 2, 40, 8, 128)
from gpu_harness import bf16_tensor, from_bf16
kt, vt, qt = bf16_tensor(k), bf16_tensor(v), bf16_tensor(q)
one, before, starts, lens = qt[:, 0].contiguous(), s.i32([0, 0]), s.i32([0, 300, 377]), s.i32(new)
pos = s.i32([range(260, 300), range(37, 77)])
out, out1 = torch.zeros_like(qt), torch.zeros_like(one)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    L.oscar_kv8_place(s.cache, kt, vt, before, starts, 300)
    L.oscar_kv8_attention(s.cache, one, lens, 400, out1, ws)
    L.oscar_kv8_attention(s.cache, qt, lens, 400, out, ws, q_pos=pos)
s.k, s.v = [k[:300], k[300:]], [v[:300], v[300:]]
for _ in range(2):
    out.zero_(), out1.zero_()
    g.replay()
    torch.cuda.synchronize()
    s.check_attention(from_bf16(out1).reshape(2, 1, 8, 128), q[:, :1])
    s.check_attention(from_bf16(out).reshape(2, 40, 8, 128), q, pos.cpu().numpy())
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.split()[-1] == "captured", r.stdout + r.stderr

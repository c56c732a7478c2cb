"""Attention over the 8-bit cache far from unit scale: values, keys and queries from 2^-100
to the largest bf16, pages of very different scales in one sequence, and logits that leave
one token.  The bounds weigh every error by the softmax weight of the token that it belongs
to, so that a page of huge values excuses nothing that it does not dominate."""
import numpy as np
import pytest

import gpu_harness as H
import kv8_harness as K
from int2_rotated_kv_gb300 import synth
from oracle import kv8

pytestmark = pytest.mark.gpu

FMTS = [kv8.INT8, kv8.E4M3]
WIDE = [0, 131072]   # see kv8_harness.Sequences.attend
BIG = float(synth.bf16_from_bits(np.array([0x7F7F], np.uint16))[0])


def bf16(x):
    """Rounded to bf16; beyond the largest finite value, to that."""
    return synth.bf16_round(np.clip(x, -BIG, BIG).astype(np.float32))


def page_max(x):
    """Largest magnitude of each token's block: its page's, or the tail's."""
    out = np.zeros(len(x))
    for p in range(0, len(x), 16):
        out[p:p + 16] = np.abs(x[p:p + 16]).max()
    return out


def check(s, got, q, pos=None):
    """Every output against fp64.  With p the softmax weights:
      logits: fp32 sums of 128 products and an offset, 24 roundings of 2^-23 of
        sum |q| 2 max|k| of the block, and 2^-21 of the logit for its scaling; an error of e
        changes p by e relative, and so the numerator and the denominator;
      weights 2^(logit + log2 s_V): ex2 and the logarithm of a scale of up to 2^121,
        2^-14; rounded to fp16, 2^-12, or by 2^-25 where the largest weight of the unit is at
        least 1: 2^-25 of max p s_V for a token, whose code is at most max|v| / s_V
        (a tail's values: at most 2^8 where s_V is a power of two, so 2^-24 of max p max|v|);
      fp32 sums: 2^-23 a page and 16 for the merges;
      the output: half a bf16 step, 2^-8."""
    m, g = got.shape[1], s.hq // s.hkv
    for b in range(s.b):
        n = len(s.k[b])
        for h in range(s.hkv):
            k, v = s.stored(b, h)
            kmax, vmax = page_max(k), page_max(v)
            for i in range(m):
                u = n if pos is None else max(0, int(pos[b, i]) + 1)
                for r in range(g):
                    row, out = q[b, i, h * g + r].astype(np.float64), got[b, i, h * g + r]
                    lg = k[:u] @ row / np.sqrt(s.d)
                    p = np.exp(lg - lg.max())
                    p /= p.sum()
                    ref, w = p @ v[:u], p @ np.abs(v[:u])
                    e = (24 * 2.0 ** -23 * np.abs(row).sum() * 2 * kmax[:u] / np.sqrt(s.d) + 2.0 ** -21 * np.abs(lg))
                    assert (p * e).sum() < 0.05                    # a bound that says something
                    tol = (2.0 ** -12 + 2.0 ** -14 + (u // 16 + 16) * 2.0 ** -23 + (p * e).sum()) * w
                    tol += (p * e) @ np.abs(v[:u]) + u * 2.0 ** -24 * (p * vmax[:u]).max()
                    assert (tol <= 0.06 * w.max()).all()
                    tol += 2.0 ** -8 * (np.abs(ref) + tol)
                    bad = ~(np.abs(out - ref) <= tol)
                    assert not bad.any(), (b, h, r, i, n, u, int(bad.sum()), out[bad][:4], ref[bad][:4], tol[bad][:4])


def rows_of(s, m):
    """The last m positions of every sequence; null for a decode step."""
    return None if m == 1 else np.stack([np.arange(x - m, x) for x in s.lens])


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("scale", [2.0 ** -95, 1e14, 1e22, 1e30])
def test_values_of_any_size(fmt, m, wide, scale):
    s = K.Sequences(3, 1, 4, 128, fmt, 700, seed=m)
    k, v = K.draw(s.rng, 645 + 320 + 151, 1, 128)
    s.place([645, 320, 151], k, bf16(v * scale))
    q = K.queries(s.rng, 3, m, 4, 128)
    pos = rows_of(s, m)
    check(s, s.attend(q, pos, wide=wide), q, pos)
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("jump", [22, 30, 60, 100])
def test_a_page_of_huge_values_that_nothing_attends_to(fmt, m, wide, jump):
    """Pages whose values are 2^jump above the others' and whose logits lie about 2^-100 below
    in weight, first, in the middle and last: they take no precision from the others."""
    s = K.Sequences(3, 1, 4, 64, fmt, 700, seed=jump)
    k, v = K.draw(s.rng, 645 + 320 + 151, 1, 64)
    k[:, :, 0] = 0
    for at in (0, 16 * 21, 645 + 16 * 19, 965 + 16 * 4):
        v[at:at + 16] *= np.float32(2.0 ** jump)
        k[at:at + 16, :, 0] = -64
    s.place([645, 320, 151], k, bf16(v))
    q = K.queries(s.rng, 3, m, 4, 64)
    q[..., 0] = 8.75
    pos = rows_of(s, m)
    check(s, s.attend(q, pos, wide=wide), q, pos)
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("up,down", [(60, -60), (119, -10), (119, -95), (100, None)])
def test_scales_far_apart_all_attended_to(fmt, m, wide, up, down):
    """Pages of 2^up among pages of 2^down (or zeros) with weights of the same order: the small
    ones' weights count in the sum though their values do not show.  The last sequence has one
    large page, and only small ones behind it."""
    s = K.Sequences(3, 1, 4, 128, fmt, 700, seed=up)
    k, v = K.draw(s.rng, 645 + 320 + 151, 1, 128)
    v = np.clip(v, -64, 64)
    small = np.arange(len(v)) // 16 % 3 > 0
    small[965:] = True
    small[965 + 32:965 + 48] = False
    v[~small] *= np.float32(2.0 ** up)
    v[small] *= np.float32(0.0 if down is None else 2.0 ** down)
    s.place([645, 320, 151], k, bf16(v))
    q = K.queries(s.rng, 3, m, 4, 128)
    pos = rows_of(s, m)
    check(s, s.attend(q, pos, wide=wide), q, pos)
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("where", ["pages", "tail"])
def test_the_largest_values_there_are(fmt, m, wide, where):
    """Values of the largest bf16, both signs, in all pages or in a tail behind ordinary ones:
    no sum of them overflows.  (All of a channel's have one sign, so the output is about as
    large, and 0.9 of the largest keeps its rounding errors finite.)"""
    s = K.Sequences(2, 1, 4, 128, fmt, 400, seed=5)
    k, v = K.draw(s.rng, 395 + 167, 1, 128)
    most = np.where(s.rng.random(128) < 0.5, -0.9 * BIG, 0.9 * BIG)
    if where == "pages":
        v[:] = bf16(most)
    else:
        v[384:395], v[395 + 160:] = bf16(most), bf16(most)
    s.place([395, 167], k, v)
    q = K.queries(s.rng, 2, m, 4, 128)
    pos = rows_of(s, m)
    if m > 1:
        pos = np.maximum(pos, np.array([[384], [160]]))
    got = s.attend(q, pos, wide=wide)
    assert np.isfinite(got).all()
    check(s, got, q, pos)
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
def test_the_largest_keys_against_tiny_queries(fmt, m, wide):
    """Keys of about the largest bf16, queries of 2^-122 to 2^-121: logits of a few units."""
    s = K.Sequences(2, 1, 4, 128, fmt, 400, seed=6)
    k, v = K.draw(s.rng, 395 + 167, 1, 128)
    k[:] = bf16(np.clip(k, -8, 8) * 2.0 ** 124)
    s.place([395, 167], k, v)
    q = bf16(s.rng.uniform(0.5, 1, (2, m, 4, 128)) * np.where(s.rng.random((2, m, 4, 128)) < 0.5, -1, 1) * 2.0 ** -121)
    pos = rows_of(s, m)
    check(s, s.attend(q, pos, wide=wide), q, pos)
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("qexp,kexp", [(13, 0), (-60, 74), (113, -97), (126, -99)])
def test_logits_that_leave_one_token(fmt, m, wide, qexp, kexp):
    """Queries of one channel, and per channel a few tokens whose keys beat all before them or
    after them by at least half a unit: a difference of 300 in the logit, so the output is that
    token's value: p s_V rounded to fp16, 2^-12, s_V itself through its logarithm, 2^-14, and the
    output to bf16, 2^-8."""
    lens = [645, 320, 151]
    s = K.Sequences(3, 1, 4, 128, fmt, 700, seed=m)
    n = sum(lens)
    _, v = K.draw(s.rng, n, 1, 128)
    k = np.zeros((n, 1, 128))
    at = 0
    for length in lens:
        k[at] = 0.5
        for c in range(128):
            t = np.sort(s.rng.choice(np.arange(1, length), 6, replace=False))
            k[at + t, 0, c] = np.arange(1, 7) if c % 2 else s.rng.permutation(np.arange(1, 7))
        at += length
    s.place(lens, bf16(k * 2.0 ** kexp), v)
    q = np.zeros((3, m, 4, 128), np.float32)
    chan = s.rng.integers(0, 128, (3, m, 4))
    np.put_along_axis(q, chan[..., None], np.float32(2.0 ** qexp), -1)
    pos = None if m == 1 else np.stack([s.rng.integers(0, x, m) for x in lens])
    got = s.attend(q, pos, wide=wide)
    for b in range(3):
        kk, vv = s.stored(b, 0)
        for i in range(m):
            u = lens[b] if pos is None else pos[b, i] + 1
            for r in range(4):
                key = kk[:u, chan[b, i, r]]
                best = int(key.argmax())
                second = np.delete(key, best).max() if u > 1 else -np.inf
                assert key[best] - second >= 0.4 * 2.0 ** kexp
                want = vv[best]
                bad = ~(np.abs(got[b, i, r] - want) <= (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -14) * 1.01 * np.abs(want))
                assert not bad.any(), (b, i, r, u, best, got[b, i, r][bad][:4], want[bad][:4])
    assert H.status(s.cache) == 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("qexp", [0, 5, 12, 16, 20, 23, 25, 40])
def test_equal_logits_however_large(fmt, m, wide, qexp):
    """All tokens have the same key, whose code times scale is exact, so all logits of a row are the
    same number, up to 2^44 and down to its negative: every weight is 1, whatever the values' scales
    (2^-20 to 2^20 from page to page), and the output is the mean.  The bound is that of `check`
    without errors of logits."""
    lens = [645, 320, 151]
    s = K.Sequences(3, 1, 4, 128, fmt, 700, seed=m + qexp)
    n = sum(lens)
    _, v = K.draw(s.rng, n, 1, 128)
    v *= np.exp2(s.rng.integers(-20, 21, n // 16 + 1).astype(np.float32))[np.arange(n) // 16][:, None, None]
    k = np.zeros((n, 1, 128), np.float32)
    k[:, :, 9] = 448 if fmt == kv8.E4M3 else 127
    s.place(lens, k, bf16(v))
    q = np.zeros((3, m, 4, 128), np.float32)
    q[..., 9] = 2.0 ** qexp * np.where(s.rng.random((3, m, 4)) < 0.3, -1, 1)
    pos = rows_of(s, m)
    got = s.attend(q, pos, wide=wide)
    for b in range(3):
        v64 = s.stored(b, 0)[1]
        vmax = page_max(v64)
        for i in range(m):
            u = lens[b] if pos is None else pos[b, i] + 1
            ref, w = v64[:u].mean(0), np.abs(v64[:u]).mean(0)
            tol = (2.0 ** -12 + 2.0 ** -14 + (u // 16 + 16) * 2.0 ** -23) * w + 2.0 ** -24 * vmax[:u].max()
            tol += 2.0 ** -8 * (np.abs(ref) + tol)
            bad = ~(np.abs(got[b, i] - ref) <= tol)
            assert not bad.any(), (b, i, u, int(bad.sum()), got[b, i][bad][:4])
    assert H.status(s.cache) == 0

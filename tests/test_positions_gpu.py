"""GPU parity of page-table extension and the rotary embedding, and a run of them
with the 8-bit cache as a serving loop uses them."""
from fractions import Fraction

import numpy as np
import pytest

import gpu_harness as H
import kv8_harness as K
from int2_rotated_kv_gb300 import synth
from oracle import kv8
from oracle import rope as orope

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ page tables

class Pages:
    def __init__(self, table, lens, free, cursor, rows, with_slots=True):
        t = H.torch()
        dev = lambda a: t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)  # noqa: E731
        b = len(lens)
        self.table, self.lens, self.free = dev(table), dev(lens), dev(free)
        self.cursor = dev([cursor])
        self.after, self.page_starts, self.row_starts = dev(np.full(b, 77)), dev(np.full(b + 1, 77)), dev(np.full(b + 1, 77))
        self.seq_ids, self.positions = dev(np.full(rows, 77)), dev(np.full(rows, 77))
        self.slots = t.full((rows,), 77, dtype=t.int64, device=H.DEV) if with_slots else None
        self.status = dev([0])
        self.dev = dev

    def step(self, new, hold=0, in_place=False):
        L = H.lib()
        L.oscar_extend_pages(self.table, self.lens, self.dev(new), self.free,
                             self.page_starts[-1:] if in_place else self.cursor,
                             self.lens if in_place else self.after, self.page_starts,
                             self.row_starts, self.seq_ids, self.positions, self.slots,
                             hold_back=hold, status=self.status)

    def got(self, in_place=False):
        H.torch().cuda.synchronize()
        out = [self.table, self.lens if in_place else self.after, self.page_starts, self.row_starts,
               self.seq_ids, self.positions] + ([self.slots] if self.slots is not None else [])
        return [x.cpu().numpy() for x in out]


def _same(got, want):
    for i, (x, y) in enumerate(zip(got, want)):
        np.testing.assert_array_equal(x, y, err_msg=f"output {i}")


@pytest.mark.parametrize("batch,hi,hold,rows", [
    (1, 1, 0, 1), (1, 5000, 15, 5000), (7, 40, 128, 300), (256, 1, 15, 256), (256, 400, 0, 60000),
    (1000, 3, 0, 3003), (2500, 2, 16, 5100), (33, 0, 0, 4), (3, 60, 1, 0)])
def test_extend_matches_the_sequential_list(batch, hi, hold, rows):
    rng = np.random.default_rng(batch + hi)
    lens, new = rng.integers(0, 700, batch), rng.integers(0, hi + 1, batch)
    maxp = -(-(700 + hi) // 16)
    held = np.array([kv8.pages_held(n, hold) for n in lens])
    table = np.full((batch, maxp), -1)
    ids = rng.permutation(held.sum() + batch * (hi // 16 + 2) + 9)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free, cursor = ids[at:], 4
    p = Pages(table, lens, free, cursor, rows)
    p.step(new, hold)
    _same(p.got(), kv8.extend(table, lens, new, free, cursor, hold, rows))
    total = int(new.sum())
    assert H.status(p) == (H.lib().DEVERR_SEQ_LEN if total > rows else 0)


@pytest.mark.parametrize("rows", [64, 5000])
def test_extend_in_place_from_a_graph(rows):
    """Lengths and cursor carried in place by a captured step, replayed."""
    t = H.torch()
    rng = np.random.default_rng(rows)
    batch, maxp, hold = 40, 20, 15
    lens = rng.integers(0, 100, batch)
    table, free = np.full((batch, maxp), -1), rng.permutation(900)
    cursor = 0
    for b in range(batch):
        for i in range(kv8.pages_held(lens[b], hold)):
            table[b, i], cursor = free[cursor], cursor + 1
    p = Pages(table, lens, free, 0, rows)
    p.page_starts[-1] = cursor
    new = p.dev(np.ones(batch))
    side = t.cuda.Stream()
    args = (p.table, p.lens, new, p.free, p.page_starts[-1:], p.lens, p.page_starts, p.row_starts,
            p.seq_ids, p.positions, p.slots)
    graph = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph, stream=side):
        H.lib().oscar_extend_pages(*args, hold_back=hold, status=p.status)
    for step in range(5):
        n = rng.integers(0, 3, batch)
        new.copy_(p.dev(n))
        graph.replay()
        want = kv8.extend(table, lens, n, free, cursor, hold, rows)
        _same(p.got(in_place=True), want)
        table, lens, cursor = want[0], want[1], int(want[2][-1])
    assert H.status(p) == 0


def test_extend_reports_what_it_refuses():
    L = H.lib()
    table = np.full((5, 4), -1)
    # negative length, negative count, one token too many for the row, and two that are fine
    lens, new = [-1, 5, 60, 63, 0], [4, -2, 5, 1, 20]
    p = Pages(table, lens, [3, 1, 4, 1, 5, 9, 2, 6], 1, 30)
    p.step(new)
    _same(p.got(), kv8.extend(table, lens, new, [3, 1, 4, 1, 5, 9, 2, 6], 1, 0, 30))
    assert H.status(p) == L.DEVERR_SEQ_LEN
    # the free list ends inside a sequence: -1, and no slot for those tokens
    p = Pages(table, [0, 0, 0, 0, 0], [7, 8, 9], 0, 200, with_slots=True)
    p.step([30, 30, 0, 16, 1])
    _same(p.got(), kv8.extend(table, [0] * 5, [30, 30, 0, 16, 1], [7, 8, 9], 0, 0, 200))
    assert H.status(p) == L.DEVERR_NO_PAGES
    # a cursor past the list: nothing left; a negative one: refused
    p = Pages(table, [0] * 5, [7, 8, 9], 50, 8)
    p.step([1, 0, 0, 0, 0])
    assert H.status(p) == L.DEVERR_NO_PAGES and p.got()[2].tolist() == [3, 4, 4, 4, 4, 4]
    p = Pages(table, [0] * 5, [7, 8, 9], -1, 8, with_slots=False)
    p.step([0, 0, 0, 0, 0])
    assert H.status(p) == L.DEVERR_SEQ_LEN
    assert (p.got()[0] == -1).all()


# ----------------------------------------------------------------------- rotary

def _phase_words(phases):
    t = H.torch()
    return t.from_numpy(phases.view(np.int64)).to(H.DEV)


def _rope_check(got, x, pos, phases, inter, amplitude=1.0, inverse=False):
    """fp32 arithmetic: cos and sin within 2^-21 (angle rounded to fp32, sincospif, the
    amplitude), two products and a sum: 2^-20 (|a| + |b|) A; rounded to bf16 once, 2^-8."""
    freq = [Fraction(int(p), 1 << 64) for p in phases]
    ref = kv8.rope(x, pos, freq, inter, amplitude, inverse)
    rd = 2 * len(freq)
    i = np.arange(rd // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    mag = np.zeros_like(ref)
    mag[..., a] = mag[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * mag
    live = np.asarray(pos) >= 0
    assert (np.abs(got - ref)[live] <= tol[live]).all()
    np.testing.assert_array_equal(got[live][..., rd:], x[live][..., rd:])


@pytest.mark.parametrize("n,hq,hkv,d,rd,inter", [
    (1, 32, 8, 128, 128, False), (37, 4, 1, 64, 64, True), (5, 3, 3, 128, 64, False),
    (9, 8, 2, 128, 40, True), (6, 2, 1, 70, 10, False), (11, 1, 0, 96, 96, False),
    (3, 0, 2, 64, 6, True), (129, 16, 2, 256, 32, False), (2, 1, 1, 2, 2, True), (41, 5, 2, 128, 74, False),
    (17, 3, 1, 64, 62, True), (7, 33, 8, 72, 26, False), (5, 2, 1, 1024, 1024, False),
    (4, 1, 1, 1024, 1022, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_matches_oracle(n, hq, hkv, d, rd, inter, in_place):
    t, L = H.torch(), H.lib()
    rng = np.random.default_rng(n + d + rd)
    phases = L.oscar_rope_phases(1e6, rd, 4.0, 32768) if d == 128 else L.oscar_rope_phases(1e4, rd)
    pos = rng.integers(0, 1 << 20, n)
    pos[0] = 0x7fffffff
    if n > 2:
        pos[1], pos[2] = 0, -1
    amplitude = 1.25 if d == 128 else 1.0
    # rows of one projection output: queries, keys, and values that stay
    x = synth.bf16_round(rng.standard_normal((n, hq + hkv + 1, d)).astype(np.float32))
    xt = H.bf16_tensor(x)
    q, k = (xt[:, :hq] if hq else None), (xt[:, hq:hq + hkv] if hkv else None)
    qo = ko = None
    if not in_place:
        qo = t.full((n, hq, d), 5.0, dtype=t.bfloat16, device=H.DEV) if hq else None
        ko = t.full((n, hkv, d), 5.0, dtype=t.bfloat16, device=H.DEV) if hkv else None
    pt = t.from_numpy(pos.astype(np.int32)).to(H.DEV)
    L.oscar_rope(q, k, pt, _phase_words(phases), qo, ko, interleaved=inter, amplitude=amplitude)
    t.cuda.synchronize()
    after = xt.float().cpu().numpy()
    for src, out, lo, hi in ((q, qo, 0, hq), (k, ko, hq, hq + hkv)):
        if src is None:
            continue
        got = after[:, lo:hi] if in_place else out.float().cpu().numpy()
        _rope_check(got.astype(np.float64), x[:, lo:hi].astype(np.float64), pos, phases, inter, amplitude)
        if n > 2:   # a padded row is left as it was
            assert (got[2] == (x[2, lo:hi] if in_place else 5.0)).all()
    np.testing.assert_array_equal(after[:, hq + hkv:] if in_place else after, x[:, hq + hkv:] if in_place else x)


def test_rope_agrees_with_the_decode_steps_embedding():
    """The half layout over the whole head is the one of oscar_decode_step_rope's oracle."""
    t, L = H.torch(), H.lib()
    rng = np.random.default_rng(1)
    x = synth.bf16_round(rng.standard_normal((50, 4, 128)).astype(np.float32))
    pos = rng.integers(0, 131072, 50)
    xt = H.bf16_tensor(x)
    L.oscar_rope(xt, None, t.from_numpy(pos.astype(np.int32)).to(H.DEV),
                 _phase_words(L.oscar_rope_phases(1e6, 128)))
    ref = orope.apply(x.transpose(1, 0, 2), pos, 1e6).transpose(1, 0, 2)
    # the fp64 angles of that oracle are off by 131072 * 2^-53 turns at most
    assert (np.abs(H.from_bf16(xt) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * 2 * np.abs(x).max()).all()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(inter):
    """The rotation is linear in x with matrix R: the gradient of sum(w * R x) is R^T w,
    the inverse call on w; against the formula, and against differences of the forward
    call (x and x + h w in bf16: h w large enough to survive the rounding)."""
    t, L = H.torch(), H.lib()
    rng = np.random.default_rng(2)
    n, h, d, rd = 20, 3, 64, 48
    phases = L.oscar_rope_phases(1e4, rd, 2.0)
    pos = rng.integers(0, 100000, n)
    pt, words = t.from_numpy(pos.astype(np.int32)).to(H.DEV), _phase_words(phases)
    w = synth.bf16_round(rng.standard_normal((n, h, d)).astype(np.float32))
    wt = H.bf16_tensor(w)
    grad = t.empty_like(wt)
    L.oscar_rope(wt, None, pt, words, grad, inverse=True, interleaved=inter, amplitude=1.5)
    _rope_check(H.from_bf16(grad), w.astype(np.float64), pos, phases, inter, 1.5, inverse=True)
    # differences: the forward map of basis-like steps, <w, R e> = <R^T w, e>
    e = synth.bf16_round(rng.standard_normal((n, h, d)).astype(np.float32))
    et = H.bf16_tensor(e)
    fwd = t.empty_like(et)
    L.oscar_rope(et, None, pt, words, fwd, interleaved=inter, amplitude=1.5)
    lhs, rhs = (w * H.from_bf16(fwd)).sum(-1), (H.from_bf16(grad) * e).sum(-1)
    # each side's values are off by half a bf16 step: 2^-8 of sum |w| |R e|, sum |R^T w| |e|
    tol = 2.0 ** -8 * 1.01 * ((np.abs(w) * np.abs(H.from_bf16(fwd))).sum(-1) +
                              (np.abs(H.from_bf16(grad)) * np.abs(e)).sum(-1)) + 1e-3 * 2.0 ** -8
    assert (np.abs(lhs - rhs) <= tol).all()


# -------------------------------------------------------- a serving loop's steps

@pytest.mark.parametrize("fmt", [kv8.INT8, kv8.E4M3])
def test_prompts_chunks_and_steps_together(fmt):
    """Page tables, rotary positions, placement and attention chained on the device for
    prompts, a chunk with its causal rows, and decode steps, with sequences that rest;
    the oracle follows from the same inputs."""
    t, L = H.torch(), H.lib()
    b, hkv, hq, d, maxp = 4, 2, 8, 128, 24
    rng = np.random.default_rng(11)
    from int2_rotated_kv_gb300 import pages
    cache = pages.allocate_kv8(b * maxp, b, maxp, hkv=hkv, hq=hq, d=d, device=H.DEV, fmt=fmt)
    free = rng.permutation(b * maxp)
    cap = 512
    p = Pages(np.full((b, maxp), -1), np.zeros(b), free, 0, cap)
    cache.page_table = p.table
    p.page_starts[-1] = 0
    phases = L.oscar_rope_phases(1e6, d, 4.0, 128)
    words = _phase_words(phases)
    freq = [Fraction(int(x), 1 << 64) for x in phases]
    model = K.Sequences(b, hkv, hq, d, fmt, 16 * maxp)
    ws = t.empty(L.oscar_kv8_workspace_size(cache, b, 40, 16 * maxp), dtype=t.uint8, device=H.DEV)
    for new in ([130, 17, 64, 0], [40, 40, 1, 0], [1, 1, 1, 1], [1, 0, 1, 1], [1, 1, 1, 0]):
        new = np.array(new)
        before = model.lens
        total = int(new.sum())
        qkv = synth.bf16_round(rng.standard_normal((cap, hq + 2 * hkv, d)).astype(np.float32))
        x = H.bf16_tensor(qkv)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        lens_before = p.lens.clone()
        p.step(new, hold=15, in_place=True)
        L.oscar_rope(q, k, p.positions, words)
        L.oscar_kv8_place(cache, k, v, lens_before, p.row_starts, int(new.max()))
        rotated = x.float().cpu().numpy()
        starts = np.concatenate([[0], np.cumsum(new)])
        pos = np.concatenate([np.arange(n0, n0 + n) for n0, n in zip(before, new)])
        ref = kv8.rope(qkv[:total, :hq + hkv], pos, freq, False)
        np.testing.assert_allclose(rotated[:total, :hq + hkv], ref, rtol=2.0 ** -8, atol=2.0 ** -17)
        np.testing.assert_array_equal(rotated[total:], qkv[total:])      # padded rows
        for i in range(b):
            rows = slice(starts[i], starts[i + 1])
            model.k[i] = np.concatenate([model.k[i], rotated[rows, hq:hq + hkv]])
            model.v[i] = np.concatenate([model.v[i], rotated[rows, hq + hkv:]])
        # rows padded to the longest chunk, positions -1 behind each sequence's own
        m = int(new.max())
        qp = np.full((b, m), -1)
        qr = np.zeros((b, m, hq, d), np.float32)
        for i in range(b):
            qp[i, :new[i]] = np.arange(before[i], before[i] + new[i])
            qr[i, :new[i]] = rotated[starts[i]:starts[i + 1], :hq]
        if m > 40:
            qp, qr, m = qp[:, -40:], qr[:, -40:], 40
        qt = H.bf16_tensor(qr if m > 1 else qr[:, 0])
        out = t.full_like(qt, float("nan"))
        qpt = t.from_numpy(np.ascontiguousarray(qp, np.int32)).to(H.DEV)
        L.oscar_kv8_attention(cache, qt, p.lens, 16 * maxp, out, ws, q_pos=qpt if m > 1 else None)
        got = H.from_bf16(out).reshape(b, m, hq, d)
        if m == 1:
            model.check_attention(got, qr)
        else:
            model.check_attention(got, qr, qp)
    np.testing.assert_array_equal(p.lens.cpu().numpy(), model.lens)
    assert H.status(cache) == 0 and H.status(p) == 0

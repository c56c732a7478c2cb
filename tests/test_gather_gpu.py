"""oscar_gather: tokens of the calibrated cache read back, against the stored codes in fp64."""
import numpy as np
import pytest

import gpu_harness as H
from int2_rotated_kv_gb300 import pages, synth
from oracle import layout

pytestmark = pytest.mark.gpu

S, W = 4, 64


def half_bits(rng, shape, lo, hi):
    return rng.uniform(lo, hi, shape).astype(np.float16).view(np.uint16)


class Model:
    """A cache whose pools hold random codes, scales, zeros and bf16 tokens (no matter where from),
    and what they stand for."""

    def __init__(self, lens, hkv, d, bits, seed=0, scale=1.0):
        self.lens, self.hkv, self.d, self.bits = np.asarray(lens), hkv, d, bits
        rng = np.random.default_rng(seed)
        self.rng = rng
        r = np.stack([np.linalg.qr(rng.standard_normal((d, d)))[0] for _ in range(2 * hkv)]).astype(np.float32)
        self.r = r.reshape(2, hkv, d, d)
        pp = pages.plan(lens, S, W, permute_seed=seed)
        clip = np.ones(hkv, np.float32)
        self.pp = pp
        self.cache = pages.allocate(pp, hkv=hkv, hq=hkv, d=d, sink=S, window=W, device=H.DEV, r_k=self.r[0],
                                    r_v=self.r[1], clip_k=clip, clip_v=clip, code_bits=bits)
        n, o, ng = pp.num_int2_pages * hkv, layout.offsets(d, bits), d // 32
        blk = rng.integers(0, 256, (n, layout.int2_block_bytes(d, bits)), dtype=np.uint8)
        sz = np.stack([half_bits(rng, (n, 16 * ng), 0.01 * scale, scale), half_bits(rng, (n, 16 * ng), -3 * scale, 0)], -1)
        blk[:, o["Ksz"]:o["Ksz"] + 2 * d] = sz.reshape(n, -1).view(np.uint8)
        blk[:, o["Vs"]:o["Vs"] + d] = half_bits(rng, (n, 16 * ng), 0.01 * scale, scale).view(np.uint8)
        blk[:, o["Vz"]:o["Vz"] + d] = half_bits(rng, (n, 16 * ng), -3 * scale, 0).view(np.uint8)
        self.blk = blk.reshape(pp.num_int2_pages, hkv, -1)
        t = H.torch()
        self.cache.int2_pool.copy_(t.from_numpy(blk.reshape(-1)))
        bf = synth.bf16_round(rng.standard_normal((pp.num_bf16_pages, hkv, 2, 16 * d)).astype(np.float32))
        self.bf = bf
        self.cache.bf16_pool.copy_(H.bf16_tensor(bf.reshape(-1)))
        # byte and bit of every code, group places
        self.at = [np.array([[f(tk, j, d) for j in range(d)] for tk in range(16)]) for f in (layout.k_code_pos, layout.v_code_pos)]
        self.el = [np.array([[f(tk, j) for j in range(d)] for tk in range(16)]) for f in (layout.bf16_k_elem, layout.bf16_v_elem)]
        self.vsz = np.array([[layout.vsz_index(tk, g, d) for g in range(ng)] for tk in range(16)])
        self.o = o

    def page(self, pid, h, kv):
        """y [16, d] of a page in fp64."""
        d, o, b = self.d, self.o, self.blk[pid, h]
        codes = np.zeros((16, d))
        base = o["Vc"] if kv else o["Kc"]
        for plane in range(self.bits // 2):
            byte = b[base + o["plane"] * plane + self.at[kv][..., 0]]
            codes = 4 * codes + ((byte >> self.at[kv][..., 1].astype(np.uint8)) & 3)
        if kv:
            s = b[o["Vs"]:o["Vs"] + d].view(np.float16)[self.vsz]
            z = b[o["Vz"]:o["Vz"] + d].view(np.float16)[self.vsz]
        else:
            sz = b[o["Ksz"]:o["Ksz"] + 2 * d].view(np.float16).reshape(16, d // 32, 2)
            s, z = sz[..., 0], sz[..., 1]
        return codes * s.astype(np.float64).repeat(32, -1) + z.astype(np.float64).repeat(32, -1)

    def tokens(self, b, h, kv):
        """x [L, d] in fp64, sum |y||R| (0 for bf16 tokens)."""
        L = int(self.lens[b])
        x, w = np.zeros((L, self.d)), np.zeros((L, self.d))
        r = self.r[kv, h].astype(np.float64)
        for p in range(-(-L // 16)):
            y = None
            for tk in range(16):
                pos = 16 * p + tk
                if pos >= L:
                    break
                if pos < S or pos >= L - W:
                    x[pos] = self.bf[self.pp.bf16_table[b, p], h, kv][self.el[kv][tk]]
                else:
                    if y is None:
                        y = self.page(self.pp.int2_table[b, p], h, kv)
                        yr, yw = y @ r.T, np.abs(y) @ np.abs(r).T
                    x[pos], w[pos] = yr[tk], yw[tk]
        return x, w

    def run(self, first, count, extra=2, max_rows=None, lens=None, stream=None):
        t = H.torch()
        starts = np.concatenate([[0], np.cumsum(count)])
        outs = [t.full((int(starts[-1]) + extra, self.hkv, self.d), 7.0, dtype=t.bfloat16, device=H.DEV) for _ in range(2)]
        i32 = lambda a: t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)  # noqa: E731
        H.lib().oscar_gather(self.cache, i32(self.lens if lens is None else lens), i32(first), i32(starts),
                             int(max(count)) if max_rows is None else max_rows, *outs, stream=stream)
        t.cuda.synchronize()
        return starts, [H.from_bf16(o) for o in outs]

    def check(self, first, count, starts, outs, heads=None):
        """The product's operands are pieces of y and R that leave 2^-16 of |y||R| (twice 2^-17), the sum
        is fp32: d additions of 2^-24 of it at most; the output is rounded to bf16 once."""
        for kv in range(2):
            for b in range(len(self.lens)):
                for h in range(self.hkv):
                    if heads is not None and (b, h) not in heads:
                        continue
                    x, w = self.tokens(b, h, kv)
                    s = slice(first[b], first[b] + count[b])
                    tol = (2.0 ** -16 + self.d * 2.0 ** -23) * w[s]
                    tol = np.where(w[s] > 0, tol + 2.0 ** -8 * (np.abs(x[s]) + tol), 0.0)
                    got = outs[kv][starts[b]:starts[b + 1], h]
                    bad = ~(np.abs(got - x[s]) <= tol)
                    assert not bad.any(), (kv, b, h, np.argwhere(bad)[:4], got[bad][:4], x[s][bad][:4])
            assert (outs[kv][starts[-1]:] == 7).all()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3), (128, 8), (64, 5)])
def test_matches_the_stored_codes(d, hkv, bits):
    """Lengths with none, one and all tokens in BF16, whole sequences and parts of them."""
    lens = [1, 3, 16, 64, 69, 70, 84, 85, 333, 700]
    m = Model(lens, hkv, d, bits, seed=d + hkv)
    first = np.array([0, 1, 0, 5, 0, 4, 15, 16, 17, 0])
    count = np.array([1, 2, 16, 0, 69, 60, 60, 69, 301, 700])
    starts, outs = m.run(first, count)
    m.check(first, count, starts, outs, heads=None if hkv < 4 else {(b, h) for b in range(10) for h in (0, hkv - 1)})
    assert H.status(m.cache) == 0


@pytest.mark.parametrize("scale", [1e-4, 1.0, 5000.0])
def test_scales(scale):
    """Zeros and scales from fp16's smallest to near its largest: y passes fp16's range."""
    m = Model([150, 260], 2, 128, 4, seed=3, scale=scale)
    first, count = np.array([0, 0]), np.array([150, 260])
    starts, outs = m.run(first, count)
    m.check(first, count, starts, outs)


def test_many_pages():
    """More tiles than the device takes at once; one long sequence beside short ones."""
    lens = [9000, 20, 1500, 0 + 1, 4000]
    m = Model(lens, 4, 128, 2, seed=5)
    first = np.array([7, 0, 0, 0, 2000])
    count = np.array([8993, 20, 1500, 1, 1999])
    starts, outs = m.run(first, count)
    m.check(first, count, starts, outs, heads={(0, 1), (1, 0), (2, 3), (3, 2), (4, 0)})
    assert H.status(m.cache) == 0


def test_after_prefill_and_appends():
    """What prefill and decode steps stored comes back as what decode attention takes it for."""
    t, L = H.torch(), H.lib()
    wl = synth.TINY
    inst = synth.draw_instance(wl, n_calib=512, with_next_token=True)
    rot = H.oracle_rotations(inst)
    cache, pp = H.make_cache(inst, rot, window=wl.window, sink=wl.sink, growth=1)
    H.prefill(cache, inst)
    n = int(inst.seq_lens[0])
    i32 = dict(dtype=t.int32, device=H.DEV)
    outs = [t.empty(n, 1, wl.head_dim, dtype=t.bfloat16, device=H.DEV) for _ in range(2)]
    L.oscar_gather(cache, t.tensor([n], **i32), t.tensor([0], **i32), t.tensor([0, n], **i32), n, *outs)
    assert H.status(cache) == 0
    k, v = (H.from_bf16(o)[:, 0] for o in outs)
    raw_k, raw_v = inst.k[0][0][:n], inst.v[0][0][:n]
    near = np.r_[0:wl.sink, n - wl.window:n]
    np.testing.assert_array_equal(k[near], raw_k[near])
    np.testing.assert_array_equal(v[near], raw_v[near])
    # attention over the rows read back, which are rounded to bf16 (2^-8 of a key: a logit is off by 2^-8
    # of sum |q||k| / sqrt d at most; the weights by twice as much), against decode's
    got = H.decode(cache, inst.q, [n])
    d = wl.head_dim
    for j in range(wl.num_q_heads):
        q = inst.q[0, j].astype(np.float64)
        lg = k @ q / np.sqrt(d)
        p = np.exp(lg - lg.max())
        p /= p.sum()
        e = 2.0 ** -8 * (np.abs(k) @ np.abs(q)) / np.sqrt(d)
        tol = (2 * (p * e).sum() + 2.0 ** -7) * (p @ np.abs(v)) + (p * e) @ np.abs(v) + H.TOL_MAX_ABS
        assert (np.abs(got[0, j] - p @ v) <= tol).all()


def test_what_it_skips_is_reported():
    t, L = H.torch(), H.lib()
    m = Model([200, 150], 2, 64, 2, seed=1)
    full = (np.array([0, 0]), np.array([200, 150]))

    def status():
        st = H.status(m.cache)
        m.cache.status.zero_()
        return st

    starts, outs = m.run(*full, max_rows=180)                        # the first asks for more
    assert status() == L.DEVERR_SEQ_LEN
    assert all((o[:200] == 7).all() for o in outs)
    m.check(np.array([0, 0]), np.array([0, 150]), np.array([200, 200, 350]), outs)
    for lens, first in (([199, 150], [0, 0]), ([200, 150], [1, 0]), ([200, 150], [-1, 0]), ([100000, 150], [0, 0])):
        starts, outs = m.run(np.array(first), full[1], lens=lens)
        assert status() == L.DEVERR_SEQ_LEN and all((o[:200] == 7).all() for o in outs)
    # page ids out of range: those tokens are left, the page's others come
    good = m.cache.int2_page_table.clone(), m.cache.bf16_page_table.clone()
    m.cache.int2_page_table[0, 2] = -1
    m.cache.int2_page_table[0, 5] = 1 << 30
    m.cache.bf16_page_table[0, 11] = m.pp.num_bf16_pages
    starts, outs = m.run(*full)
    assert status() == L.DEVERR_PAGE_ID
    gone = np.r_[32:48, 80:96, 176:192]
    for kv in range(2):
        assert (outs[kv][gone] == 7).all()
        for h in range(2):
            x, w = m.tokens(0, h, kv)
            rest = np.setdiff1d(np.arange(200), gone)
            tol = np.where(w > 0, 2.0 ** -15 * w + 2.0 ** -8 * (np.abs(x) + 2.0 ** -15 * w), 0)
            assert (np.abs(outs[kv][:200, h] - x) <= tol)[rest].all()
    m.cache.int2_page_table.copy_(good[0]), m.cache.bf16_page_table.copy_(good[1])
    starts, outs = m.run(*full)
    m.check(*full, starts, outs)
    assert status() == 0
    with pytest.raises(ValueError):
        bad = m.cache.bf16_page_table
        m.cache.bf16_page_table = bad[:, :-1].contiguous()
        try:
            m.run(*full)
        finally:
            m.cache.bf16_page_table = bad
    x = t.zeros(3, 2, 64, dtype=t.bfloat16, device=H.DEV)
    i = t.zeros(3, dtype=t.int32, device=H.DEV)
    for args in ((i[:2], i[:2], i, 3, x[:, :1], x), (i[:2], i[:1], i, 3, x, x), (i[:2], i[:2], i, 3, x, x.float()),
                 (i[:2].cpu(), i[:2], i, 3, x, x), (i, i, t.zeros(4, dtype=t.int32, device=H.DEV), 3, x, x)):
        with pytest.raises(ValueError):
            L.oscar_gather(m.cache, *args)


def test_streams_and_graphs():
    t, L = H.torch(), H.lib()
    m = Model([500, 311], 3, 128, 4, seed=8)
    full = (np.array([0, 11]), np.array([500, 300]))
    starts, want = m.run(*full)
    m.check(*full, starts, want, heads={(0, 0), (1, 2)})
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    _, got = m.run(*full, stream=stream)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    i32 = dict(dtype=t.int32, device=H.DEV)
    lens, first, rows = t.tensor([500, 311], **i32), t.tensor([0, 11], **i32), t.tensor([0, 500, 800], **i32)
    outs = [t.full((802, 3, 128), 7.0, dtype=t.bfloat16, device=H.DEV) for _ in range(2)]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        L.oscar_gather(m.cache, lens, first, rows, 500, *outs)
    graph.replay()
    t.cuda.synchronize()
    for a, b in zip(outs, want):
        np.testing.assert_array_equal(H.from_bf16(a), b)
    first.copy_(t.tensor([100, 0], **i32))
    rows.copy_(t.tensor([0, 400, 700], **i32))
    for o in outs:
        o.fill_(7.0)
    graph.replay()
    t.cuda.synchronize()
    m.check(np.array([100, 0]), np.array([400, 300]), np.array([0, 400, 700]), [H.from_bf16(o) for o in outs],
            heads={(0, 1), (1, 0)})


def test_offsets_beyond_4_gib():
    t = H.torch()
    m = Model([200], 8, 128, 4, seed=2)
    size = 8 * layout.int2_block_bytes(128, 4)
    need = (5 << 30) // size
    pool = t.empty(need * size, dtype=t.uint8, device=H.DEV)
    ids = m.cache.int2_page_table[0].cpu().numpy()
    old = m.cache.int2_pool.view(-1, size)
    new = ids.copy()
    for p, pid in enumerate(ids):
        if pid >= 0:
            new[p] = need - 1 - 7 * p
            pool.view(-1, size)[int(new[p])] = old[int(pid)]
    m.cache.int2_pool = pool
    m.cache.int2_page_table.copy_(t.from_numpy(new[None]))
    starts, outs = m.run(np.array([0]), np.array([200]))
    m.check(np.array([0]), np.array([200]), starts, outs, heads={(0, 0), (0, 7)})


def test_a_bound_of_rows_that_says_nothing():
    """max_rows of all that an int32 holds: the rows that there are bound the work."""
    m = Model([500], 2, 64, 2, seed=6)
    full = np.array([7]), np.array([493])
    starts, outs = m.run(*full, max_rows=(1 << 31) - 1)
    m.check(*full, starts, outs)
    assert int(m.cache.status.item()) == 0


def test_rotations_written_just_before():
    """Codes turned back by the rotations that the stream's call before has put there."""
    t = H.torch()
    m = Model([300], 2, 128, 4, seed=9)
    full = np.array([0]), np.array([300])
    old = m.r.copy()
    for turn in range(3):
        m.r = np.ascontiguousarray(np.roll(old, turn + 1, axis=-1))
        new = [t.from_numpy(x).to(H.DEV) for x in m.r]
        m.cache.r_k.copy_(new[0].view_as(m.cache.r_k)), m.cache.r_v.copy_(new[1].view_as(m.cache.r_v))
        starts, outs = m.run(*full)
        m.check(*full, starts, outs)


def test_refuses_rotations_and_pools():
    t, L = H.torch(), H.lib()
    m = Model([40], 2, 64, 2, seed=3)
    x = t.zeros(40, 2, 64, dtype=t.bfloat16, device=H.DEV)
    lens, zero, rows = (t.tensor(a, dtype=t.int32, device=H.DEV) for a in ([40], [0], [0, 40]))
    for name, bad in (("r_k", m.cache.r_k.bfloat16()), ("r_v", m.cache.r_v.flatten()[:-1].clone()),
                      ("r_k", m.cache.r_k.cpu()), ("bf16_pool", m.cache.bf16_pool.float())):
        good = getattr(m.cache, name)
        setattr(m.cache, name, bad)
        with pytest.raises(ValueError):
            L.oscar_gather(m.cache, lens, zero, rows, 40, x, x.clone())
        setattr(m.cache, name, good)

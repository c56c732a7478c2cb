"""oscar_gather over what prefill and decode steps have stored, for sinks and windows of other sizes; beside other calls
on other streams."""
import numpy as np
import pytest

import gpu_harness as H
import kv4_harness as K4
import kv8_harness as K8
from int2_rotated_kv_gb300 import pages, synth
from oracle import cache as ocache, layout, quant

pytestmark = pytest.mark.gpu


class Stored:
    """Sequences of random tokens, lens[b] of them placed by a prefill and `steps` more by appends."""

    def __init__(self, lens, steps, hkv, d, bits, sink, window, seed=0, clips=True):
        t, L = H.torch(), H.lib()
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens) + steps
        self.hkv, self.d, self.bits, self.sink, self.window = hkv, d, bits, sink, window
        self.r = np.stack([np.linalg.qr(rng.standard_normal((d, d)))[0]
                           for _ in range(2 * hkv)]).astype(np.float32).reshape(2, hkv, d, d)
        self.pp = pages.plan(lens, sink, window, growth=steps, permute_seed=seed)
        high = np.full(hkv, 1e4, np.float32)   # clips nothing
        self.cache = pages.allocate(self.pp, hkv=hkv, hq=hkv, d=d, sink=sink, window=window, device=H.DEV,
                                    r_k=self.r[0], r_v=self.r[1], clip_k=high, clip_v=high, code_bits=bits)
        self.x = [[synth.bf16_round(rng.standard_normal((n, hkv, d)).astype(np.float32)) for n in self.lens]
                  for _ in range(2)]
        i32 = lambda a: t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)  # noqa: E731
        first = [H.bf16_tensor(np.concatenate([x[:n] for x, n in zip(self.x[kv], lens)])) for kv in range(2)]
        L.oscar_prefill_quantize(self.cache, *first, i32(np.repeat(np.arange(len(lens)), lens)),
                                 i32(np.concatenate([np.arange(n) for n in lens])), i32(lens))
        for i in range(steps):
            new = [H.bf16_tensor(np.stack([x[n + i] for x, n in zip(self.x[kv], lens)])) for kv in range(2)]
            L.oscar_quantize_append(self.cache, *new, i32(np.asarray(lens) + i + 1))
        if not clips:   # whoever reads need not have them
            self.cache.clip_k = self.cache.clip_v = None
        self.pools = H.pools(self.cache)
        assert H.status(self.cache) == 0

    def read(self, first, count, stream=None, outs=None):
        t = H.torch()
        starts = np.concatenate([[0], np.cumsum(count)])
        if outs is None:
            outs = [t.full((int(starts[-1]), self.hkv, self.d), 7.0, dtype=t.bfloat16, device=H.DEV) for _ in range(2)]
        i32 = lambda a: t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)  # noqa: E731
        args = [i32(self.lens), i32(first), i32(starts)]
        if stream is not None:
            stream.wait_stream(t.cuda.current_stream())
        H.lib().oscar_gather(self.cache, *args, int(max(count)), *outs, stream=stream)
        return starts, outs, args

    def check(self, first, count, starts, outs):
        """Against the codes that the pools hold, as in test_gather_gpu.py (pieces leave 2^-16 of |y||R|, the sum d
        roundings of 2^-24 of it at most, then bf16), and against the tokens themselves: a code is off by half a scale,
        and by the fp16 roundings of zero and scale, 2^-11 of |min| and of max - min, 3 * 2^-11 max|y| at most; the
        rotation adds 2^-12 |x|, of which its fp32 sums need little.  R is orthogonal: so much in length."""
        d, got2, gotb = self.d, *self.pools
        size, sizeb = layout.int2_block_bytes(d, self.bits), layout.bf16_block_bytes(d) // 2
        outs = [H.from_bf16(o) for o in outs]
        seen = [0, 0]
        for b, L in enumerate(self.lens):
            coded = ocache.is_int2(np.arange(L), L, self.sink, self.window)
            for h in range(self.hkv):
                for pg in range(first[b] // 16, -(-(first[b] + count[b]) // 16) if count[b] else 0):
                    pos = np.arange(max(16 * pg, first[b]), min(16 * pg + 16, first[b] + count[b]))
                    for mine in (coded[pos], ~coded[pos]):
                        if not mine.any():
                            continue
                        slot = pos[mine] - 16 * pg
                        is_code = bool(coded[pos[mine][0]])
                        pid = int((self.pp.int2_table if is_code else self.pp.bf16_table)[b, pg])
                        at = (pid * self.hkv + h) * (size if is_code else sizeb)
                        block = (layout.unpack_int2_block(got2[at:at + size], d, self.bits) if is_code
                                 else layout.unpack_bf16_block(gotb[at:at + sizeb], d))
                        for kv in range(2):
                            got = outs[kv][starts[b] + pos[mine] - first[b], h]
                            raw = self.x[kv][b][pos[mine], h].astype(np.float64)
                            seen[is_code] += len(slot)
                            if not is_code:
                                np.testing.assert_array_equal(got, synth.bf16_from_bits(block[kv][slot]))
                                np.testing.assert_array_equal(got, raw)
                                continue
                            c, s, z = (block[3 * kv + i][slot] for i in range(3))
                            y, r = quant.dequantize(c, s, z), self.r[kv, h].astype(np.float64)
                            x, w = y @ r.T, np.abs(y) @ np.abs(r).T
                            tol = (2.0 ** -16 + d * 2.0 ** -23) * w
                            assert (np.abs(got - x) <= tol + 2.0 ** -8 * (np.abs(x) + tol)).all(), (kv, b, h, pg)
                            full = raw @ r
                            off = (s.astype(np.float64) / 2).repeat(32, -1) + 3 * 2.0 ** -11 * np.abs(
                                full.reshape(len(slot), -1, 32)).max(-1).repeat(32, -1)
                            far = (np.linalg.norm(off, axis=-1) + 2.0 ** -12 * np.linalg.norm(raw, axis=-1)
                                   + np.linalg.norm(2.0 ** -8 * np.abs(got) + tol, axis=-1))
                            assert (np.linalg.norm(got - raw, axis=-1) <= far).all(), (kv, b, h, pg)
        return seen


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("d,hkv,sink,window", [(64, 2, 4, 64), (128, 3, 0, 1), (128, 1, 20, 300), (64, 1, 37, 16),
                                               (128, 2, 130, 17)])
def test_tokens_of_prefill_and_appends(d, hkv, bits, sink, window):
    """Sinks of none, of several pages and of more than a tile; windows of one token, beside a page's border, and of more
    than a tile; sequences that are shorter than both."""
    steps = 23
    lens = [1, 10, 40, 150, 333, 700]
    m = Stored(lens, steps, hkv, d, bits, sink, window, seed=d + window, clips=bits == 2)
    whole = np.zeros(6, int), m.lens
    starts, outs, _ = m.read(*whole)
    plain, coded = m.check(*whole, starts, outs)
    part = np.array([0, 3, 17, 64, 131, 5]), np.array([24, 0, 30, 100, 200, 718])
    m.check(*part, *m.read(*part)[:2])
    assert plain and coded and H.status(m.cache) == 0


def test_beside_other_calls_on_other_streams():
    """Two streams read the same cache back, a third has attention in tiles of 128 columns, which takes all of tensor
    memory too, a fourth a prefill's rotation: each gives what it gives alone."""
    t, L = H.torch(), H.lib()
    m = Stored([900, 31, 2000], 3, 4, 128, 4, 4, 64, seed=1)
    small = Stored([400, 77], 2, 2, 64, 2, 4, 64, seed=2)
    whole, ends = (np.zeros(3, int), m.lens), (np.array([0, 5]), small.lens - 5)
    _, want, _ = m.read(*whole)
    _, want_small, _ = small.read(*ends)
    s = K4.Sequences(2, 2, 8, 128, 3000, seed=3)
    s.place([3000, 1203])
    rows = 70
    q = K8.queries(s.rng, 2, rows, 8, 128)
    pos = s.lens[:, None] - rows + np.arange(rows)
    want_rows = s.attend(q, pos)
    qt, lens, pt = H.bf16_tensor(q), s.i32(s.lens), s.i32(pos)
    ws = t.zeros(L.oscar_kv4_workspace_size(s.cache, 2, rows, 3000), dtype=t.uint8, device=H.DEV)
    k, v = (H.bf16_tensor(np.concatenate(x)) for x in m.x)
    i32 = lambda a: t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)  # noqa: E731
    sid, at, final = i32(np.repeat(np.arange(3), m.lens)), i32(np.concatenate([np.arange(n) for n in m.lens])), i32(m.lens)
    other = pages.allocate(m.pp, hkv=4, hq=4, d=128, sink=4, window=64, device=H.DEV, r_k=m.r[0], r_v=m.r[1],
                           clip_k=np.full(4, 1e4, np.float32), clip_v=np.full(4, 1e4, np.float32), code_bits=4)
    L.oscar_prefill_quantize(other, k, v, sid, at, final)
    want_pools = H.pools(other)
    streams = [t.cuda.Stream() for _ in range(4)]
    outs = [[t.full_like(x, 7.0) for x in want] for _ in range(2)]
    outs_small = [t.full_like(x, 7.0) for x in want_small]
    out_rows = t.full_like(qt, float("nan"))
    other.int2_pool.zero_(), other.bf16_pool.zero_()
    args = [i32(a) for a in (m.lens, whole[0], np.concatenate([[0], np.cumsum(whole[1])]))]
    args_small = [i32(a) for a in (small.lens, ends[0], np.concatenate([[0], np.cumsum(ends[1])]))]
    t.cuda.synchronize()
    for _ in range(12):
        for i in range(2):
            L.oscar_gather(m.cache, *args, int(m.lens.max()), *outs[i], stream=streams[i])
        L.oscar_kv4_attention(s.cache, qt, lens, 3000, out_rows, ws, q_pos=pt, stream=streams[2])
        L.oscar_prefill_quantize(other, k, v, sid, at, final, stream=streams[3])
        L.oscar_gather(small.cache, *args_small, int(ends[1].max()), *outs_small, stream=streams[3])
    t.cuda.synchronize()
    for got in outs:
        assert all(t.equal(a, b) for a, b in zip(got, want))
    assert all(t.equal(a, b) for a, b in zip(outs_small, want_small))
    np.testing.assert_array_equal(H.from_bf16(out_rows).reshape(want_rows.shape), want_rows)
    for a, b in zip(H.pools(other), want_pools):
        np.testing.assert_array_equal(a, b)
    assert all(H.status(c) == 0 for c in (m.cache, small.cache, s.cache, other))

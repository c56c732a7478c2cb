"""A model of sequences in an 8-bit cache for the GPU tests: raw tokens on the host,
the library's cache beside them, and what the oracle says of both."""
import numpy as np

import gpu_harness as H
from int2_rotated_kv_gb300 import pages, synth
from oracle import kv8

NAN_PATTERN = 0xA5   # pools start with this byte, so that untouched bytes show


def draw(rng, n, hkv, d, scale=1.0):
    """bf16 keys and values [n, hkv, d]: channel spreads, four strong key channels."""
    sk, sv = (np.exp(0.5 * rng.standard_normal((hkv, d))) for _ in range(2))
    off = np.zeros((hkv, d))
    for h in range(hkv):
        c = rng.choice(d, 4, replace=False)
        sk[h, c] *= 15
        off[h, c] = 3
    k = synth.bf16_round((scale * (rng.standard_normal((n, hkv, d)) * sk + off)).astype(np.float32))
    v = synth.bf16_round((scale * rng.standard_normal((n, hkv, d)) * sv).astype(np.float32))
    return k, v


class Sequences:
    def __init__(self, batch, hkv, hq, d, fmt, max_len, seed=0, spare=3, permute_tails=False):
        t = H.torch()
        self.b, self.hkv, self.hq, self.d, self.fmt = batch, hkv, hq, d, fmt
        self.rng = np.random.default_rng(seed)
        self.max_pages = max(1, max_len // 16)
        total = batch * self.max_pages + spare
        self.cache = pages.allocate_kv8(total, batch, self.max_pages, hkv=hkv, hq=hq, d=d,
                                        device=H.DEV, fmt=fmt, num_tails=batch + spare)
        self.ids = self.rng.permutation(total)
        self.table = self.ids[:batch * self.max_pages].reshape(batch, self.max_pages).astype(np.int32)
        self.cache.page_table.copy_(t.from_numpy(self.table))
        self.cache.pool.fill_(NAN_PATTERN)
        self.cache.tail.view(t.uint8).fill_(0xFF)        # NaN
        self.tail_ids = np.arange(batch)
        if permute_tails:
            self.tail_ids = self.rng.permutation(batch + spare)[:batch]
            self.cache.tail_ids = t.from_numpy(self.tail_ids.astype(np.int32)).to(H.DEV)
        self.k = [np.zeros((0, hkv, d), np.float32) for _ in range(batch)]
        self.v = [np.zeros((0, hkv, d), np.float32) for _ in range(batch)]

    @property
    def lens(self):
        return np.array([len(x) for x in self.k])

    def i32(self, a):
        t = H.torch()
        return t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)

    def place(self, new, k=None, v=None, stream=None, extra_rows=0, packed=False, max_new=None):
        """Appends new[b] tokens to each sequence, on both sides."""
        new = np.asarray(new)
        n = int(new.sum())
        if k is None:
            k, v = draw(self.rng, n + extra_rows, self.hkv, self.d)
        starts = np.concatenate([[0], np.cumsum(new)])
        kt, vt = H.bf16_tensor(k), H.bf16_tensor(v)
        if packed:   # columns of one projection output
            t = H.torch()
            both = t.cat([t.zeros_like(kt), kt, vt], 1).contiguous()
            kt, vt = both[:, self.hkv:2 * self.hkv], both[:, 2 * self.hkv:]
        H.lib().oscar_kv8_place(self.cache, kt, vt, self.i32(self.lens), self.i32(starts),
                                int(max(new.max(), 1)) if max_new is None else max_new, stream=stream)
        for b in range(self.b):
            self.k[b] = np.concatenate([self.k[b], k[starts[b]:starts[b + 1]]])
            self.v[b] = np.concatenate([self.v[b], v[starts[b]:starts[b + 1]]])

    def stored(self, b, h):
        """Values that the cache stands for: keys, values [L, d]."""
        return kv8.stored(self.k[b][:, h], self.fmt), kv8.stored(self.v[b][:, h], self.fmt)

    def check_pools(self):
        """Every byte of the pool, and every tail slot that holds a token."""
        H.torch().cuda.synchronize()
        d, order = self.d, kv8.orders(self.d)
        want = np.full((self.cache.pool.shape[0], self.hkv, 32 * d + 16), NAN_PATTERN, np.uint8)
        tail = self.cache.tail.float().cpu().numpy()
        for b in range(self.b):
            for h in range(self.hkv):
                for kv, x in enumerate((self.k[b][:, h], self.v[b][:, h])):
                    for p in range(len(x) // 16):
                        scale, codes = kv8.block(x[16 * p:16 * p + 16], self.fmt)
                        blk = want[self.table[b, p], h]
                        blk[16 * d * kv:16 * d * (kv + 1)][order[kv]] = codes
                        blk[32 * d:].view(np.float32)[kv::2] = [scale, 0]
                    rest = x[len(x) // 16 * 16:]
                    got = tail[self.tail_ids[b], h, kv][order[kv][:len(rest)]]
                    np.testing.assert_array_equal(got, rest)
        got = self.cache.pool.cpu().numpy()
        bad = np.argwhere(got != want)
        assert len(bad) == 0, (len(bad), bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])

    def attend(self, q, q_pos=None, max_len=None, lens=None, ws=None, stream=None, wide=0):
        """The library's output as float64, [B, M, Hq, d] (M = 1 for a decode step).
        wide: with a page table of that many columns, and lengths up to it announced: what
        the library takes for a long context, and tiles of 128 query columns for."""
        t, L = H.torch(), H.lib()
        if wide:
            table = self.cache.page_table
            self.cache.page_table = t.full((self.b, wide), -1, dtype=t.int32, device=H.DEV)
            self.cache.page_table[:, :self.max_pages] = table
            if q_pos is not None and q_pos.shape[1] * self.hq // self.hkv > 8:
                size = L.oscar_kv8_workspace_size(self.cache, self.b, q_pos.shape[1], 16 * wide)
                assert size > 5 << 20   # partial results of 128 columns
            try:
                return self.attend(q, q_pos, 16 * wide, lens, ws, stream)
            finally:
                self.cache.page_table = table
        lens = self.lens if lens is None else np.asarray(lens)
        m = 1 if q_pos is None else q_pos.shape[1]
        max_len = max(1, int(lens.max())) if max_len is None else max_len
        qt = H.bf16_tensor(q if q_pos is not None else q[:, 0])
        out = t.full_like(qt, float("nan"))
        if ws is None:
            size = L.oscar_kv8_workspace_size(self.cache, len(lens), m, max_len)
            assert size > 0
            ws = t.full((size,), 0xFF, dtype=t.uint8, device=H.DEV)
        L.oscar_kv8_attention(self.cache, qt, self.i32(lens), max_len, out, ws,
                              q_pos=None if q_pos is None else self.i32(q_pos), stream=stream)
        t.cuda.synchronize()
        return H.from_bf16(out).reshape(len(lens), m, self.hq, self.d)

    def check_attention(self, got, q, q_pos=None, lens=None, drop=(), heads=None):
        """Every output element against fp64, within the bound of the kernel's arithmetic.

        Errors, relative to w = sum p |v|: p s_V rounded to fp16 (2^-12), a logit off by
        e changes p by 2 e at most (numerator and denominator): fp32 sums of 128 products
        and an offset of 128 sum q, 8 + 16 additions of 2^-23 of sum |q| 255 s_K (e4m3:
        448) and 2^-21 of the logit itself for its scaling; ex2 and fp32 sums 2^-18; weights
        below 2^-31 of the largest value scale are lost: 2^-30 max|v| per token at most.  The
        sum over pages takes one fp32 addition per page of a warp's share (n / 16 at most)
        and 16 for the merges, each off by 2^-23 of w at most.  The output is rounded to
        bf16 once: half a step, 2^-8."""
        lens = self.lens if lens is None else lens
        m, g = got.shape[1], self.hq // self.hkv
        top = 448 if self.fmt == kv8.E4M3 else 255
        for b in range(len(lens)):
            n = int(lens[b])
            for h in range(self.hkv):
                if heads is not None and (b, h) not in heads:
                    continue
                k, v = (x[:n] for x in self.stored(b, h))
                keep = np.ones(n, bool)
                for p in drop:
                    keep[16 * p:16 * p + 16] = False
                kept = np.flatnonzero(keep)
                sk = np.abs(k[np.isfinite(k)]).max() if np.isfinite(k).any() else 0.0
                for i in range(m):
                    limit = n if q_pos is None else max(0, min(int(q_pos[b, i]) + 1, n))
                    if q_pos is not None and q_pos[b, i] >= n:
                        limit = 0
                    for r in range(g):
                        row = q[b, i, h * g + r].astype(np.float64)
                        u = int((kept < limit).sum())
                        ref, w = kv8.attention(row, k[keep], v[keep], u)
                        out = got[b, i, h * g + r]
                        if not np.isfinite(ref).all():
                            assert not np.isfinite(out[~np.isfinite(ref)]).any()
                            assert (np.isfinite(out) == np.isfinite(ref)).all()
                            continue
                        s = sk / (448 if self.fmt == kv8.E4M3 else 127)
                        e = (24 * 2.0 ** -23 * np.abs(row).sum() * top * s +
                             2.0 ** -21 * (np.abs(k[keep][:u] @ row).max() if u else 0)) / np.sqrt(self.d)
                        tol = (2.0 ** -12 + 2 * e + 2.0 ** -18 + (u // 16 + 16) * 2.0 ** -23) * w
                        tol += 2.0 ** -30 * u * (np.abs(v[keep][:u]).max() if u else 0)
                        tol += 2.0 ** -8 * (np.abs(ref) + tol)
                        bad = ~(np.abs(out - ref) <= tol)
                        assert not bad.any(), (b, h, r, i, n, limit, out[bad][:4], ref[bad][:4], tol[bad][:4])


def queries(rng, b, m, hq, d, scale=1.0):
    decay = 0.9 ** (0.5 * np.arange(d))
    return synth.bf16_round((scale * rng.standard_normal((b, m, hq, d)) * decay).astype(np.float32))

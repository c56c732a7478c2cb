"""Sequences in a 4-bit cache for the GPU tests: kv8_harness's model with the 4-bit calls and
oracle.  Its bounds hold as they stand: code * s is exact where the 8-bit cache has codes, and
an e4m3 code times its scale reaches the block's largest magnitude as code * s * g does."""
import numpy as np

import gpu_harness as H
import kv8_harness as K
from int2_rotated_kv_gb300 import pages
from oracle import kv4, kv8

NAN_PATTERN = K.NAN_PATTERN


class Sequences(K.Sequences):
    def __init__(self, batch, hkv, hq, d, max_len, seed=0, spare=3, permute_tails=False):
        t = H.torch()
        self.b, self.hkv, self.hq, self.d, self.fmt = batch, hkv, hq, d, kv8.E4M3
        self.rng = np.random.default_rng(seed)
        self.max_pages = max(1, max_len // 16)
        total = batch * self.max_pages + spare
        self.cache = pages.allocate_kv4(total, batch, self.max_pages, hkv=hkv, hq=hq, d=d,
                                        device=H.DEV, num_tails=batch + spare)
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
        self._stored = {}

    def place(self, new, k=None, v=None, stream=None, extra_rows=0, packed=False, max_new=None):
        """Appends new[b] tokens to each sequence, on both sides."""
        new = np.asarray(new)
        n = int(new.sum())
        if k is None:
            k, v = K.draw(self.rng, n + extra_rows, self.hkv, self.d)
        starts = np.concatenate([[0], np.cumsum(new)])
        kt, vt = H.bf16_tensor(k), H.bf16_tensor(v)
        if packed:   # columns of one projection output
            t = H.torch()
            both = t.cat([t.zeros_like(kt), kt, vt], 1).contiguous()
            kt, vt = both[:, self.hkv:2 * self.hkv], both[:, 2 * self.hkv:]
        H.lib().oscar_kv4_place(self.cache, kt, vt, self.i32(self.lens), self.i32(starts),
                                int(max(new.max(), 1)) if max_new is None else max_new, stream=stream)
        for b in range(self.b):
            self.k[b] = np.concatenate([self.k[b], k[starts[b]:starts[b + 1]]])
            self.v[b] = np.concatenate([self.v[b], v[starts[b]:starts[b + 1]]])
        self._stored = {}

    def stored(self, b, h):
        if (b, h) not in self._stored:
            self._stored[b, h] = kv4.stored(self.k[b][:, h], False), kv4.stored(self.v[b][:, h], True)
        return self._stored[b, h]

    def check_pools(self):
        """Every byte of the pool, and every tail slot that holds a token."""
        H.torch().cuda.synchronize()
        d, order = self.d, kv8.orders(self.d)
        want = np.full((self.cache.pool.shape[0], self.hkv, 18 * d + 16), NAN_PATTERN, np.uint8)
        tail = self.cache.tail.float().cpu().numpy()
        for b in range(self.b):
            for h in range(self.hkv):
                k, v = self.k[b][:, h], self.v[b][:, h]
                for p in range(len(k) // 16):
                    want[self.table[b, p], h] = kv4.block_bytes(k[16 * p:16 * p + 16], v[16 * p:16 * p + 16])
                for kv, x in enumerate((k, v)):
                    rest = x[len(x) // 16 * 16:]
                    got = tail[self.tail_ids[b], h, kv][order[kv][:len(rest)]]
                    np.testing.assert_array_equal(got, rest)
        got = self.cache.pool.cpu().numpy()
        bad = np.argwhere(got != want)
        assert len(bad) == 0, (len(bad), bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])

    def attend(self, q, q_pos=None, max_len=None, lens=None, ws=None, stream=None, wide=0):
        """The library's output as float64, [B, M, Hq, d] (M = 1 for a decode step).  wide: with a
        page table of that many columns, and lengths up to it announced."""
        t, L = H.torch(), H.lib()
        if wide:
            table = self.cache.page_table
            self.cache.page_table = t.full((self.b, wide), -1, dtype=t.int32, device=H.DEV)
            self.cache.page_table[:, :self.max_pages] = table
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
            size = L.oscar_kv4_workspace_size(self.cache, len(lens), m, max_len)
            assert size > 0
            ws = t.full((size,), 0xFF, dtype=t.uint8, device=H.DEV)
        L.oscar_kv4_attention(self.cache, qt, self.i32(lens), max_len, out, ws,
                              q_pos=None if q_pos is None else self.i32(q_pos), stream=stream)
        t.cuda.synchronize()
        return H.from_bf16(out).reshape(len(lens), m, self.hq, self.d)

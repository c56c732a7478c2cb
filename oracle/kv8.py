"""8-bit cache oracle: block codes, block layout, attention over the values that the
cache stands for, and the page bookkeeping of a step.

One scale per block of 16 tokens x one KV head (keys and values apart).  With a the
largest finite magnitude of the block,
    scale = fl32(a / top), inv = fl32(top / a), code = round(fl32(x inv)),
top = 127 (codes integers, stored plus 128) or 448 (codes e4m3, ties to even); a block
with a < 2^-100 is zeros; NaN -> 0, infinities -> +-top.  Products and quotients of
the definition are rounded once to fp32: formed in fp64 (exact products, quotients
whose second rounding is innocuous) and rounded.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
INT8, E4M3 = 0, 1


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 byte (NaN for 0x7f and 0xff)."""
    out = np.zeros(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = np.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -v if s else v
    return out


_E4M3 = e4m3_values()


def _e4m3_bytes(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte, ties to the even mantissa, |y| <= 480."""
    mag = _E4M3[:127]                                   # ascending, 0 .. 448
    i = np.clip(np.searchsorted(mag, np.abs(y)), 1, 126)
    lo, hi = mag[i - 1], mag[i]
    a = np.abs(y)
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return (np.where(up, i, i - 1) | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def block(x: np.ndarray, fmt: int):
    """(scale float32, bytes uint8 [16, d]) of one block x [16, d] of bf16 values."""
    x = np.asarray(x, np.float64)
    top = 448.0 if fmt == E4M3 else 127.0
    finite = np.isfinite(x)
    a = np.abs(x[finite]).max() if finite.any() else 0.0
    if not a >= 2.0 ** -100:
        return np.float32(0), np.full(x.shape, 0 if fmt == E4M3 else 128, np.uint8) | (
            np.where(np.signbit(x) & ~np.isnan(x), 128, 0).astype(np.uint8) if fmt == E4M3 else 0)
    scale, inv = np.float32(a / top), np.float32(top / a)
    y = (np.where(finite, x, 0.0) * np.float64(inv)).astype(np.float32).astype(np.float64)
    y = np.where(np.isposinf(x), top, np.where(np.isneginf(x), -top, y))
    y = np.where(np.isnan(x), 0.0, y)
    return scale, _e4m3_bytes(y) if fmt == E4M3 else (np.rint(y) + 128).astype(np.uint8)


def values(scale, codes: np.ndarray, fmt: int) -> np.ndarray:
    c = _E4M3[codes] if fmt == E4M3 else codes.astype(np.float64) - 128.0
    return c * np.float64(scale)


def key_element(t: int, c: int) -> int:
    """Element of (token, channel) in a key area, by the layout's formula."""
    return (((c // 64) * 2 + t % 2) * 32 + 4 * (t // 2) + (c // 16) % 4) * 16 + c % 16


def value_element(t: int, c: int) -> int:
    return ((c // 32) * 32 + 4 * ((c // 4) % 8) + t // 4) * 16 + 4 * (c % 4) + t % 4


def orders(d: int):
    """(key, value) element indices [16, d]."""
    return (np.array([[key_element(t, c) for c in range(d)] for t in range(PAGE)]),
            np.array([[value_element(t, c) for c in range(d)] for t in range(PAGE)]))


def stored(x: np.ndarray, fmt: int) -> np.ndarray:
    """The values that the cache stands for, of one head's tokens x [L, d]: whole pages
    coded, the rest as it is."""
    out = np.asarray(x, np.float64).copy()
    for p in range(len(x) // PAGE):
        s = slice(p * PAGE, (p + 1) * PAGE)
        out[s] = values(*block(x[s], fmt), fmt)
    return out


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, limit: int):
    """softmax(q k^T / sqrt d) v over tokens 0 .. limit - 1 (zeros when there are none);
    also sum p |v|, which the error of rounded weights is measured by."""
    d = q.shape[-1]
    if limit <= 0:
        return np.zeros(d), np.zeros(d)
    w = k[:limit] @ q / np.sqrt(d)
    w = np.exp(w - w.max())
    w /= w.sum()
    return w @ v[:limit], w @ np.abs(v[:limit])


def pages_held(n: int, hold: int) -> int:
    return max(0, -(-(n - hold) // PAGE))


def extend(table, lens, new, free, cursor, hold, max_rows):
    """One step of page bookkeeping, sequence by sequence (see oscar_extend_pages)."""
    table = np.array(table)
    seq_ids, positions = (np.full(max_rows, -1, np.int64) for _ in range(2))
    slots = np.full(max_rows, -1, np.int64)
    page_starts, row_starts, after = [cursor], [0], []
    row = 0
    for b, (n0, n) in enumerate(zip(lens, new)):
        if n0 < 0 or n < 0 or n0 + n - hold > table.shape[1] * PAGE:
            n = 0
        lo, hi = pages_held(n0, hold), pages_held(n0 + n, hold)
        for p in range(lo, hi):
            table[b, p] = free[cursor] if cursor < len(free) else -1
            cursor += 1
        for t in range(n0, n0 + n):
            if row < max_rows:
                seq_ids[row], positions[row] = b, t
                if t // PAGE < hi and table[b, t // PAGE] >= 0:
                    slots[row] = int(table[b, t // PAGE]) * PAGE + t % PAGE
            row += 1
        after.append(n0 + n)
        page_starts.append(cursor)
        row_starts.append(row)
    return table, np.array(after), np.array(page_starts), np.array(row_starts), seq_ids, positions, slots


def rope(x: np.ndarray, positions, freq: np.ndarray, interleaved: bool, amplitude: float = 1.0,
         inverse: bool = False) -> np.ndarray:
    """Rotates x [n, heads, d]; freq [rd / 2] turns per token (python floats or Fractions
    of full precision are reduced modulo one turn before rounding)."""
    x = np.asarray(x, np.float64)
    half = len(freq)
    turns = np.array([[float((int(m) * f) % 1) for f in freq] for m in positions])
    ang = 2 * np.pi * turns * (-1 if inverse else 1)
    c, s = amplitude * np.cos(ang)[:, None], amplitude * np.sin(ang)[:, None]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y

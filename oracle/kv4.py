"""4-bit cache oracle: codes and scales of a page, the block's bytes, and the values that the
cache stands for.

With a the largest finite magnitude of the 16 x d keys (or values) of a page and KV head, m that
of a block of 16 (keys: a channel's 16 tokens; values: 16 channels of a token),
    g = fl32(a / 2688), s = e4m3(fl32(m fl32(448 / a))),
    code = e2m1(fl32(x fl32(fl32(2688 / a) / s))),
nearest, ties to even, codes saturating at 6; s = 0 or a < 2^-97: zeros; NaN -> 0, an infinity ->
+-a.  A value is code * s * g.  Quotients and products of the definition are rounded once to
fp32: formed in fp64 (exact products, quotients whose second rounding is innocuous) and rounded.
"""
from __future__ import annotations

import numpy as np

from . import kv8

PAGE = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def e2m1_codes(y: np.ndarray) -> np.ndarray:
    """Nearest e2m1 code, ties to the even code, saturating; bit 3 is the sign."""
    a = np.minimum(np.abs(y), 6.0)
    i = np.clip(np.searchsorted(E2M1, a), 1, 7)
    lo, hi = E2M1[i - 1], E2M1[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return (np.where(up, i, i - 1) | np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def e2m1_values(codes: np.ndarray) -> np.ndarray:
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def block(x: np.ndarray, value: bool):
    """(g float32, scale bytes, codes uint8 [16, d]) of keys or values x [16, d] (bf16 values);
    scale bytes [1, d] for keys, [16, d/16] for values."""
    x = np.asarray(x, np.float64)
    d = x.shape[1]
    finite = np.isfinite(x)
    a = np.abs(x[finite]).max() if finite.any() else 0.0
    live = a >= 2.0 ** -97
    x = np.where(np.isposinf(x), a, np.where(np.isneginf(x), -a, np.where(np.isnan(x), 0.0, x)))
    to_block, to_code = (_f32(448.0 / a), _f32(2688.0 / a)) if live else (0.0, 0.0)
    m = np.abs(x).reshape(16, d // 16, 16).max(-1) if value else np.abs(x).max(0, keepdims=True)
    scales = kv8._e4m3_bytes(_f32(m * to_block))
    s = kv8.e4m3_values()[scales]
    r = np.where(s > 0, _f32(to_code / np.where(s > 0, s, 1.0)), 0.0)
    r = np.repeat(r, 16, -1) if value else np.broadcast_to(r, x.shape)
    return np.float32(a / 2688.0 if live else 0.0), scales, e2m1_codes(_f32(x * r))


def values(g, scales: np.ndarray, codes: np.ndarray, value: bool) -> np.ndarray:
    s = kv8.e4m3_values()[scales]
    s = np.repeat(s, 16, -1) if value else s
    return e2m1_values(codes) * s * np.float64(g)


def key_nibble(t: int, c: int) -> int:
    """Index of a key's code among the nibbles of the key codes, low nibble of a byte first."""
    return 2 * (((c // 64) * 32 + 4 * (t // 2) + (c // 16) % 4) * 16 + 8 * (t % 2) + (c % 16) // 2) + c % 2


def value_nibble(t: int, c: int) -> int:
    return 2 * (((c // 64) * 32 + 4 * ((c // 4) % 8) + t // 4) * 16 + 8 * ((c // 32) % 2) + 2 * (c % 4)
                + (t % 4) // 2) + t % 2


def value_scale_byte(t: int, b: int) -> int:
    return (b // 4) * 64 + ((b % 2) * 4 + t // 4) * 8 + ((b // 2) % 2) * 4 + t % 4


def orders(d: int):
    """(key, value) nibble indices [16, d], value-scale byte indices [16, d/16]."""
    return (np.array([[key_nibble(t, c) for c in range(d)] for t in range(PAGE)]),
            np.array([[value_nibble(t, c) for c in range(d)] for t in range(PAGE)]),
            np.array([[value_scale_byte(t, b) for b in range(d // 16)] for t in range(PAGE)]))


def block_bytes(k: np.ndarray, v: np.ndarray) -> np.ndarray:
    """The 18 d + 16 bytes of a page's keys and values [16, d]."""
    d = k.shape[1]
    ko, vo, so = orders(d)
    out = np.zeros(18 * d + 16, np.uint8)
    scale = np.zeros(4, np.float32)
    for which, (x, order) in enumerate(((k, ko), (v, vo))):
        scale[which], scales, codes = block(x, which == 1)
        nib = np.zeros(16 * d, np.uint8)
        nib[order] = codes
        out[8 * d * which:8 * d * (which + 1)] = nib[0::2] | (nib[1::2] << 4)
        if which == 0:
            out[16 * d:17 * d] = scales[0]
        else:
            out[17 * d:18 * d][so] = scales
    out[18 * d:] = scale.view(np.uint8)
    return out


def stored(x: np.ndarray, value: bool) -> np.ndarray:
    """The values that the cache stands for, of one head's keys or values x [L, d]: whole pages
    coded, the rest as it is."""
    out = np.asarray(x, np.float64).copy()
    for p in range(len(x) // PAGE):
        s = slice(p * PAGE, (p + 1) * PAGE)
        out[s] = values(*block(x[s], value), value)
    return out

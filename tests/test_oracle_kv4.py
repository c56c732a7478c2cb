"""Pins of the 4-bit cache oracle: e2m1 rounding, scales and codes of a page, the order of its
bytes."""
import numpy as np
import pytest

from int2_rotated_kv_gb300 import synth
from oracle import kv4, kv8


def test_e2m1_rounding():
    both = np.concatenate([kv4.E2M1, -kv4.E2M1])
    np.testing.assert_array_equal(kv4.e2m1_codes(both), np.arange(16))
    np.testing.assert_array_equal(kv4.e2m1_values(np.arange(16, dtype=np.uint8)), both)
    # ties to the even code, and beyond the largest
    y = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -5.0, -100.0])
    np.testing.assert_array_equal(kv4.e2m1_values(kv4.e2m1_codes(y)),
                                  [0, 1, 1, 2, 2, 4, 4, 6, 0, -4, -6])
    y = np.random.default_rng(0).uniform(-6, 6, 1000)
    err = np.abs(kv4.e2m1_values(kv4.e2m1_codes(y)) - y)
    assert (err <= np.maximum(0.25, np.abs(y) / 5)).all()


@pytest.mark.parametrize("value", [False, True])
def test_scales_and_codes(value):
    rng = np.random.default_rng(1)
    x = synth.bf16_round((rng.standard_normal((16, 64)) * np.exp(rng.standard_normal(64))).astype(np.float32))
    g, scales, codes = kv4.block(x, value)
    a = np.abs(x).max()
    assert g == np.float32(a / 2688) and scales.shape == ((16, 4) if value else (1, 64))
    y = kv4.values(g, scales, codes, value)
    m = np.abs(x).reshape(16, 4, 16).max(-1).repeat(16, -1) if value else np.abs(x).max(0, keepdims=True)
    # a step between codes is at most a third of the scale's top; the scale is off by 2^-4 of itself
    # at most (and nothing here lies among its subnormal values), so values saturate by as much
    assert (np.abs(y - x) <= m / 6 * (1 + 2.0 ** -4) + 2.0 ** -20 * a).all()
    # the block of the largest value has the largest scale, and stands for it
    assert scales.max() == 0x7e
    i = np.unravel_index(np.abs(x).argmax(), x.shape)
    assert y[i] == pytest.approx(x[i], rel=2.0 ** -22)
    x[3, 5], x[4, 6], x[9, 0] = np.nan, np.inf, -np.inf
    y = kv4.values(*kv4.block(x, value), value)
    big = np.abs(x[np.isfinite(x)]).max()
    assert y[3, 5] == 0 and y[4, 6] == pytest.approx(big) and y[9, 0] == pytest.approx(-big)
    for small in (0.0, 2.0 ** -98):
        g, scales, codes = kv4.block(np.full((16, 64), small), value)
        assert g == 0 and not scales.any() and not codes.any()
    # a block that is nothing beside the page's largest value has scale 0
    x = np.full((16, 64), 1.0)
    x[:, 16:32] = 2.0 ** -30
    g, scales, codes = kv4.block(x, value)
    assert not kv4.values(g, scales, codes, value)[:, 16:32].any()


@pytest.mark.parametrize("d", [64, 128])
def test_order_of_bytes(d):
    keys, values, scales = kv4.orders(d)
    for order in (keys, values):
        np.testing.assert_array_equal(np.sort(order.ravel()), np.arange(16 * d))
    np.testing.assert_array_equal(np.sort(scales.ravel()), np.arange(d))
    # chunks of 16 bytes: two tokens of 16 channels; four tokens of 4 channels and of those 32 further
    t, c = np.unravel_index(np.argsort(keys.ravel()), keys.shape)
    t, c = t.reshape(-1, 2, 16), c.reshape(-1, 2, 16)
    assert (t == t[:, :1, :1] + np.arange(2)[:, None]).all() and (c == c[:, :1, :1] + np.arange(16)).all()
    t, c = np.unravel_index(np.argsort(values.ravel()), values.shape)
    t, c = t.reshape(-1, 2, 4, 4), c.reshape(-1, 2, 4, 4)
    assert (t == t[:, :1, :1, :1] + np.arange(4)).all()
    assert (c == c[:, :1, :1, :1] + np.arange(2)[:, None, None] * 32 + np.arange(4)[:, None]).all()
    # a page's bytes read back by the formulas
    rng = np.random.default_rng(2)
    k, v = (synth.bf16_round(rng.standard_normal((16, d)).astype(np.float32)) for _ in range(2))
    blk = kv4.block_bytes(k, v)
    g, s, codes = kv4.block(v, True)
    nib = np.stack([blk[8 * d:16 * d] & 15, blk[8 * d:16 * d] >> 4], -1).ravel()
    np.testing.assert_array_equal(nib[values], codes)
    np.testing.assert_array_equal(blk[17 * d:18 * d][scales], s)
    assert blk[18 * d:].view(np.float32)[1] == g and not blk[18 * d + 8:].any()
    assert np.abs(kv4.stored(np.concatenate([k, k[:3]]), False)[16:] - k[:3]).max() == 0


def test_four_bits_say_what_they_should():
    """Relative error of a page of normal values: e2m1 with a scale for 16 of them keeps about 0.1;
    a key channel that is larger than the others takes nothing from them."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((16, 128))
    for value in (False, True):
        y = kv4.stored(synth.bf16_round(x.astype(np.float32)), value)
        assert np.linalg.norm(y - x) < 0.12 * np.linalg.norm(x)
    x[:, 5] *= 30
    y = kv4.stored(synth.bf16_round(x.astype(np.float32)), False)
    rest = np.arange(128) != 5
    assert np.linalg.norm((y - x)[:, rest]) < 0.12 * np.linalg.norm(x[:, rest])
    assert kv8.stored(x, kv8.INT8).shape == y.shape

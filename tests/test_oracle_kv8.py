"""Pins of the 8-bit cache oracle: e4m3 values and rounding, block codes, the layout's
element order, page bookkeeping."""
import numpy as np
import pytest

from int2_rotated_kv_gb300 import synth
from oracle import kv8


def test_e4m3_values_and_rounding():
    v = kv8.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7e] == 448.0 and v[0x01] == 2.0 ** -9 and v[0xb8] == -1.0
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff])
    finite = v[np.isfinite(v)]
    np.testing.assert_array_equal(v[kv8._e4m3_bytes(finite)], finite)   # fixed points
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 0.01,
                        (finite[:126] + finite[1:127]) / 2]).astype(np.float32)   # with all midpoints
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(kv8._e4m3_bytes(y.astype(np.float64)), want)


@pytest.mark.parametrize("fmt", [kv8.INT8, kv8.E4M3])
def test_block_codes(fmt):
    rng = np.random.default_rng(1)
    x = synth.bf16_round(rng.standard_normal((16, 64)).astype(np.float32) * 3)
    scale, codes = kv8.block(x, fmt)
    y = kv8.values(scale, codes, fmt)
    # half a step of the code (int8: of the block, e4m3: relative, 2^-4), and the fp32
    # roundings of inv, x inv and scale: 2^-24 of the value each
    top = 448.0 if fmt else 127.0
    step = 0.5 * scale if fmt == kv8.INT8 else np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)
    assert (np.abs(y - x) <= step + np.abs(x) * 2.0 ** -22).all()
    assert np.abs(y).max() == pytest.approx(np.abs(x).max(), rel=2.0 ** -22)
    assert scale == np.float32(np.abs(x).max() / top)
    x[3, 5], x[4, 6], x[9, 0] = np.nan, np.inf, -np.inf
    scale, codes = kv8.block(x, fmt)
    y = kv8.values(scale, codes, fmt)
    big = np.abs(x[np.isfinite(x)]).max()
    assert y[3, 5] == 0 and y[4, 6] == pytest.approx(big) and y[9, 0] == pytest.approx(-big)
    for small in (0.0, 2.0 ** -101):
        scale, codes = kv8.block(np.full((16, 64), small), fmt)
        assert scale == 0 and (kv8.values(scale, codes, fmt) == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_layout_is_a_bijection_in_16_byte_chunks(d):
    for order, same in zip(kv8.orders(d), ("token", "square")):
        np.testing.assert_array_equal(np.sort(order.ravel()), np.arange(16 * d))
        t, c = np.unravel_index(np.argsort(order.ravel()), order.shape)
        t, c = t.reshape(d, 16), c.reshape(d, 16)           # one row per 16-byte chunk
        if same == "token":
            assert (t == t[:, :1]).all() and (c == c[:, :1] + np.arange(16)).all()
        else:
            assert (t == t[:, :1] + np.tile(np.arange(4), 4)).all()
            assert (c == c[:, :1] + np.repeat(np.arange(4), 4)).all()


def test_attention_and_stored():
    rng = np.random.default_rng(2)
    k, v, q = rng.standard_normal((40, 8)), rng.standard_normal((40, 8)), rng.standard_normal(8)
    o, a = kv8.attention(q, k, v, 3)
    w = np.exp(k[:3] @ q / np.sqrt(8))
    np.testing.assert_allclose(o, (w[:, None] * v[:3]).sum(0) / w.sum(), rtol=1e-12)
    assert (a >= np.abs(o)).all()
    assert (kv8.attention(q, k, v, 0)[0] == 0).all()
    x = synth.bf16_round(rng.standard_normal((37, 64)).astype(np.float32))
    s = kv8.stored(x, kv8.INT8)
    assert (s[32:] == x[32:]).all() and (s[:32] != x[:32]).any()


def test_extend():
    t = np.full((2, 4), -1)
    t[0, 0] = 9
    got = kv8.extend(t, [16, 0], [1, 33], [5, 6, 7, 8], 0, 0, 40)
    assert got[0].tolist() == [[9, 5, -1, -1], [6, 7, 8, -1]]
    assert got[1].tolist() == [17, 33] and got[2].tolist() == [0, 1, 4] and got[3].tolist() == [0, 1, 34]
    assert got[6][0] == 5 * 16 and got[6][33] == 8 * 16 and got[6][34] == -1
    assert kv8.pages_held(15, 15) == 0 and kv8.pages_held(16, 15) == 1 and kv8.pages_held(17, 15) == 1

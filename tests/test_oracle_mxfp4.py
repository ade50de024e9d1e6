"""Pins of oracle/mxfp4.py: the E2M1 table, ties and saturation by hand, the
block rule's invariants, packing, and the product against one dense matmul."""

import numpy as np
import pytest

from oracle import gateup, mxfp4


def test_e2m1_table():
    assert mxfp4.e2m1_value(np.arange(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert mxfp4.e2m1_value(np.arange(8, 16)).tolist() == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert np.array_equal(mxfp4.e2m1_code(mxfp4.e2m1_value(np.arange(16))), np.arange(16))


def test_ties_go_to_the_even_code():
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert mxfp4.e2m1_code(ties).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert mxfp4.e2m1_code([-t for t in ties]).tolist() == [8, 10, 10, 12, 12, 14, 14]
    eps = 1e-9
    assert mxfp4.e2m1_code([t - eps for t in ties]).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert mxfp4.e2m1_code([t + eps for t in ties]).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert mxfp4.e2m1_code([6.0, 7.99, 1e30, -1e30]).tolist() == [7, 7, 7, 15]


def test_hand_block():
    x = np.zeros((1, 32))
    x[0, :5] = [7.0, -5.0, 0.25, -0.0, 3.0]       # top 7 -> exponent floor(log2 7) - 2 = 0
    codes, s = mxfp4.quantize(x)
    assert s.tolist() == [[127]]
    assert (codes[0, 0] & 15, codes[0, 0] >> 4) == (7, 14)     # 6 (saturated), -4 (tie to even)
    assert (codes[0, 1] & 15, codes[0, 1] >> 4) == (0, 8)      # 0 (tie to even), -0
    assert codes[0, 2] & 15 == 5


@pytest.mark.parametrize("shift", [-140, -126, -20, 0, 60, 120])
def test_block_rule(shift):
    rng = np.random.default_rng(3)
    x = np.ldexp(rng.standard_normal((40, 96)), shift)
    codes, s = mxfp4.quantize(x)
    v = mxfp4.dequantize(codes, s)
    b, w = x.reshape(40, 3, 32), v.reshape(40, 3, 32)
    top = np.abs(b).max(-1)
    scale = np.ldexp(1.0, s.astype(int) - 127)
    free = s > 0                                          # the exponent is not clamped
    assert np.all(top[free] >= 4 * scale[free]) and np.all(top < 8 * scale)
    # half a step of the grid at most, or the saturation of (6, 8)
    err = np.abs(b - w)
    step = np.where(np.abs(b) < 2 * scale[..., None], 0.5, np.where(np.abs(b) < 4 * scale[..., None], 1.0, 2.0))
    assert np.all(err <= step * scale[..., None] / 2 * np.where(np.abs(b) > 6 * scale[..., None], 2, 1))
    again = mxfp4.quantize(v)
    assert np.array_equal(mxfp4.dequantize(*again), v)    # quantised values are kept


def test_special_blocks():
    x = np.ones((1, 128))
    x[0, 3], x[0, 40] = np.inf, np.nan
    x[0, 64:96] = 0.0
    codes, s = mxfp4.quantize(x)
    assert s[0].tolist()[:3] == [255, 255, 0]
    assert not codes[0, :48].any()
    v = mxfp4.dequantize(codes, s)
    assert np.isnan(v[0, :64]).all() and not v[0, 64:96].any() and (v[0, 96:] == 1).all()


def test_grouped_is_a_dense_product_and_combine_by_hand():
    rng = np.random.default_rng(4)
    E, R, K, P = 3, 8, 64, 7
    codes, s = mxfp4.quantize(rng.standard_normal((E, R, K)))
    x = mxfp4.dequantize(*mxfp4.quantize(rng.standard_normal((P, K))))
    off = np.array([0, 2, 2, 7])
    y, mag = mxfp4.grouped(x, codes, s, off)
    w = mxfp4.dequantize(codes, s)
    for r in range(P):
        e = 0 if r < 2 else 2
        want = [sum(x[r, k] * w[e, n, k] for k in range(K)) for n in range(R)]
        assert np.allclose(y[r], want, rtol=1e-14, atol=0)
        assert np.all(mag[r] >= np.abs(y[r]))
    sub, _ = mxfp4.grouped(x, codes, s, off, rows=[6, 0])
    assert np.array_equal(sub, y[[6, 0]])
    # the other oracle's form of the GELU cancels for large negative gates: compared near zero
    small = y / np.abs(y).max()
    act, _ = mxfp4.gelu_tanh_act(small)
    assert np.allclose(act, gateup.epilogue(small), rtol=1e-13, atol=0)
    out, m = mxfp4.combine(y, np.array([[0.25, 0.75]]), np.array([3, 1]))
    assert np.allclose(out[0], 0.25 * y[3] + 0.75 * y[1]) and np.all(m >= np.abs(out) - 1e-12)

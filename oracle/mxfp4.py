"""MXFP4 quantiser and the grouped MXFP4 products (fp64).

Test infrastructure: only the tests use this module; the GPU path never does.

OCP Microscaling Formats (MX) specification v1.0: blocks of 32 values along K
share an E8M0 scale 2^(s - 127) (s = 255: NaN); the values are E2M1, sign /
two exponent bits (bias 1) / one mantissa bit. The conversion takes the
exponent of the block's largest magnitude less that of E2M1's largest binade
(2), rounds to nearest with ties to even and saturates. Readings:
  * the scale's exponent is at least -127 (an all-zero block too: s = 0);
  * a block with an infinity or NaN gets s = 255 and codes 0;
  * two codes a byte, the lower index in the low nibble.
"""

import numpy as np

BLOCK = 32


def e2m1_value(code):
    """The value of 4-bit codes, from the fields."""
    code = np.asarray(code, dtype=np.int64)
    sign = np.where(code & 8, -1.0, 1.0)
    ex, man = (code >> 1) & 3, code & 1
    mag = np.where(ex == 0, 0.5 * man, np.ldexp(1.0 + 0.5 * man, ex - 1))
    return sign * mag


def e2m1_code(v):
    """Nearest E2M1 code of finite v, ties to the even code, saturating."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 7.0)[..., None]            # everything above 6 is 6
    grid = e2m1_value(np.arange(8))
    dist = np.abs(a - grid)
    best = dist.min(-1, keepdims=True)
    near = dist == best                                  # one code, or two in a tie
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True) & (near.sum(-1, keepdims=True) > 1), even, near)
    return pick.argmax(-1) + 8 * np.signbit(v)


def quantize(x):
    """x [..., K] fp64 -> (codes uint8 [..., K/2], scales uint8 [..., K/32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    _, ex = np.frexp(np.where(bad, 1.0, top))            # top = m 2^ex, m in [0.5, 1)
    e = np.where(top > 0, np.maximum(ex - 1 - 2, -127), -127)
    y = np.where(bad[..., None], 0.0, np.ldexp(np.where(bad[..., None], 0.0, b), -e[..., None]))
    code = e2m1_code(y)
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def dequantize(codes, scales):
    """codes [..., K/2], scales [..., K/32] -> fp64 [..., K] (NaN where s = 255)."""
    codes = np.asarray(codes, dtype=np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    s = np.repeat(np.asarray(scales, dtype=np.int64), BLOCK, axis=-1)
    return np.where(s == 255, np.nan, np.ldexp(e2m1_value(c), s - 127))


def grouped(xq, codes, scales, expert_off, rows=None):
    """rows of xq [P, K] (fp64 values, expert order) times their expert's
    weights: fp64 [P or len(rows), R], and the sums of the terms' magnitudes."""
    P, R = xq.shape[0], codes.shape[1]
    rows = np.arange(P) if rows is None else np.asarray(rows)
    y, mag = np.zeros((len(rows), R)), np.zeros((len(rows), R))
    e_of = np.searchsorted(np.asarray(expert_off), rows, side="right") - 1
    for e in np.unique(e_of):
        w = dequantize(codes[e], scales[e])
        i = np.nonzero(e_of == e)[0]
        y[i] = xq[rows[i]] @ w.T
        mag[i] = np.abs(xq[rows[i]]) @ np.abs(w).T
    return y, mag


def gelu_tanh_act(gu):
    """gelu_tanh(gate) * up of [.., N] rows (gate half, then up half), and |z|.

    v/2 (1 + tanh z) as v / (1 + exp(-2z)), the same function: 1 + tanh z
    cancels to nothing in fp64 for z below about -18."""
    half = gu.shape[-1] // 2
    g, u = gu[..., :half], gu[..., half:]
    z = np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-2.0 * z)) * u, np.abs(z)


def combine(y, topk_w, pair_pos):
    """out[t] = sum_j w[t, j] y[pair_pos[t k + j]] and the sum of the terms' magnitudes."""
    T, k = topk_w.shape
    g = y[np.asarray(pair_pos).reshape(T, k)]
    w = np.asarray(topk_w, dtype=np.float64)[..., None]
    return (w * g).sum(1), np.abs(w * g).sum(1)

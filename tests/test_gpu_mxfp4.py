"""GPU parity: the MXFP4 quantiser, grouped gate_up and grouped down projection
against oracle/mxfp4.py.

Tolerances, all from counts of roundings (2^-24 = half a float32 step):
  * quantiser and inverse: bit-exact (every step is exact but the rounding to
    E2M1, whose ties are unique).
  * gate_up and y where every term is a multiple of a unit and the terms'
    magnitudes sum to less than 2^24 units (asserted per case): every partial
    sum is a float32 number, so the result is exact whatever the order.
  * elsewhere: K additions, each off by at most a float32 step of the terms'
    magnitude sum: K 2^-23 sum|terms|.
  * act from the kernel's own gate_up sums g, u: z and the exponent take 6
    roundings and 6 rounded constants (12 |z| 2^-24 relative in exp(-2z)), the
    exponential and reciprocal 2 steps each, the sum, two products 1 each: (12 |z| + 8) 2^-24
    relative, and 2^-124 |g u| where the exponential leaves float32's normal
    range. A bf16 act adds half a bf16 step, 2^-8 relative.
  * out: topk products and additions, (topk + 1) 2^-24 sum|w y| on top of y's own.
"""

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
import synth
from oracle import mxfp4, numfmt, router
from tests.gpu_util import bf16_cuda

pytestmark = pytest.mark.gpu


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).cuda()


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


# ----------------------------------------------------------------------------------------------------- quantiser

def _special_rows():
    rng = np.random.default_rng(11)
    x = rng.standard_normal((24, 96)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 1e-38                                           # subnormal neighbours, the clamped scale
    x[3] *= 3e-45
    x[4] *= 1e37
    x[5, 7] = np.inf
    x[6, 40] = np.nan
    x[7, 95] = -np.inf
    x[8, :32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4) * np.tile([1, -1, 1, -1], 8)
    x[8, 32:64] = x[8, :32] * 2.0 ** -60
    x[9] = np.where(rng.random(96) < 0.5, 2.0 ** -127, -(2.0 ** -126))
    x[10, :32] = 0.0
    x[10, 3] = 7.9999
    x[11] = np.float32(3.3895314e38)                        # the largest bf16
    x[12, ::32] = 1e30                                      # one large value a block
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 2048), (257, 160), (64, 4096)])
def test_quantiser_random(gpu_available, dtype, rows, K):
    print(f"quantise {rows} x {K} {dtype}", flush=True)
    rng = np.random.default_rng(rows * K)
    x = torch.from_numpy((rng.standard_normal((rows, K)) * 2.0 ** rng.integers(-30, 30, (rows, 1))).astype(np.float32))
    x = x.to(dtype)
    _check_quantiser(x)


def _check_quantiser(x):
    codes, scales = i8h.mxfp4_quantize(x.cuda())
    want_c, want_s = mxfp4.quantize(values(x))
    torch.cuda.synchronize()
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    want = mxfp4.dequantize(want_c, want_s)
    for dt in (torch.float32, torch.bfloat16):
        got = i8h.mxfp4_dequantize(codes, scales, dtype=dt)
        assert got.dtype == dt
        expect = torch.from_numpy(want).float().to(dt)        # 6 * 2^126 and more is infinite in either type
        g, w = got.float().cpu().numpy(), expect.float().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(w))
        keep = ~np.isnan(w)
        assert np.array_equal(g[keep], w[keep]) and np.array_equal(np.signbit(g[keep]), np.signbit(w[keep]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantiser_special_values(gpu_available, dtype):
    print(f"quantise special values {dtype}", flush=True)
    _check_quantiser(torch.from_numpy(_special_rows()).to(dtype))


def test_inverse_of_every_code_and_scale(gpu_available):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    print("dequantise all codes x all scales", flush=True)
    with np.errstate(over="ignore"):
        want = mxfp4.dequantize(codes, scales)
        for dt in (torch.float32, torch.bfloat16):
            got = i8h.mxfp4_dequantize(u8(codes), u8(scales), dtype=dt)
            w = torch.from_numpy(want).float().to(dt).float().numpy()
            assert np.array_equal(got.float().cpu().numpy(), w, equal_nan=True)


def test_quantiser_shapes(gpu_available):
    x = torch.randn((2, 3, 64), device="cuda")
    codes, scales = i8h.mxfp4_quantize(x)
    assert codes.shape == (2, 3, 32) and scales.shape == (2, 3, 2)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    assert i8h.mxfp4_quantize(x, codes=c2, scales=s2)[0] is c2
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    out = torch.empty((2, 3, 64), dtype=torch.bfloat16, device="cuda")
    assert i8h.mxfp4_dequantize(codes, scales, out=out) is out
    empty = i8h.mxfp4_quantize(torch.empty((0, 64), device="cuda"))
    assert empty[0].shape == (0, 32) and i8h.mxfp4_dequantize(*empty).shape == (0, 64)


# -------------------------------------------------------------------------------------------------------- products

def _weights(rng, E, R, K, spread):
    codes = rng.integers(0, 256, (E, R, K // 2), dtype=np.uint8)
    return codes, (120 + rng.integers(0, spread + 1, (E, R, K // 32))).astype(np.uint8)


def _act_bound(want, z, g, u):
    return (12 * z + 8) * 2.0 ** -24 * np.abs(want) + 2.0 ** -124 * np.abs(g * u)


def _units(x_scales, w_scales):
    """The smallest unit that every term is a multiple of: half of half, at the smallest scales."""
    return 0.25 * 2.0 ** (int(x_scales.min()) - 127 + int(w_scales.min()) - 127)


def _routing(T, E, topk, seed, bias=None):
    rng = np.random.default_rng(seed)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    if bias is not None:
        lg = (lg + np.asarray(bias, dtype=np.float32)).astype(np.float32)
    return router.route(lg, topk)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _gpu_routing(r):
    return {"topk_ids": _i32(r["ids"]), "topk_w": torch.from_numpy(np.asarray(r["weights"], dtype=np.float32)).cuda(),
            "expert_off": _i32(r["expert_off"]), "sorted_pairs": _i32(r["sorted_pairs"]), "pair_pos": _i32(r["pair_pos"])}


def _check_gateup(T, K, E, topk, N, seed, spread=2, wide=0, bias=None, rows=None):
    """wide: octaves between the tokens' blocks; 0 keeps the sums exact."""
    rng = np.random.default_rng(seed)
    r = _routing(T, E, topk, seed, bias)
    # blocks whose largest value lies in [4, 8): every block has the same scale, or `wide` octaves more or less
    x = rng.standard_normal((T, K)).clip(-3, 3) * 2
    x.reshape(T, -1, 32)[:, :, 0] = 4.5
    x *= np.repeat(2.0 ** rng.integers(-wide, wide + 1, (T, K // 32)), 32, axis=1) if wide else 1.0
    xb = synth.to_bf16_bits(x.astype(np.float32))
    codes, scales = _weights(rng, E, N, K, spread)
    gr = _gpu_routing(r)
    print(f"gate_up T={T} K={K} E={E} topk={topk} N={N} wide={wide}", flush=True)
    xt, ct, st = bf16_cuda(xb), u8(codes), u8(scales)
    gu, act = i8h.moe_gateup_mxfp4_grouped(xt, ct, st, topk, gr["expert_off"], gr["sorted_pairs"])
    _, a16 = i8h.moe_gateup_mxfp4_grouped(xt, ct, st, topk, gr["expert_off"], gr["sorted_pairs"], gate_up=False,
                                          act_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    qc, qs = mxfp4.quantize(numfmt.bf16_from_bits(xb))
    xq = mxfp4.dequantize(qc, qs)[np.asarray(r["sorted_pairs"]) // topk]
    ref, mag = mxfp4.grouped(xq, codes, scales, r["expert_off"], rows=rows)
    sel = slice(None) if rows is None else rows
    got = gu.cpu().numpy().astype(np.float64)[sel]
    if wide == 0:
        assert mag.max() < 2.0 ** 24 * _units(qs, scales)
        assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    else:
        assert np.all(np.abs(got - ref) <= K * 2.0 ** -23 * mag)
    want, z = mxfp4.gelu_tanh_act(got)
    half = N // 2
    a = act.cpu().numpy().astype(np.float64)[sel]
    lim = _act_bound(want, z, got[:, :half], got[:, half:])
    assert np.all(np.abs(a - want) <= lim)
    assert torch.equal(a16, act.to(torch.bfloat16))          # the float32 value rounded to nearest even
    return r


GATEUP = [
    (1, 128, 1, 1, 64), (1, 2048, 128, 8, 1536), (2, 384, 8, 2, 128), (3, 640, 5, 3, 192),
    (7, 1920, 60, 4, 1408), (8, 256, 4, 4, 64), (16, 1152, 3, 1, 320), (33, 2048, 2, 1, 128),
    (64, 128, 16, 8, 256), (65, 256, 1, 1, 64), (128, 512, 128, 8, 192), (129, 896, 7, 2, 448),
    (200, 384, 1, 1, 128), (300, 256, 3, 2, 576), (512, 640, 9, 3, 128), (700, 128, 2, 2, 64),
]


@pytest.mark.parametrize("T,K,E,topk,N", GATEUP)
def test_gate_up(gpu_available, T, K, E, topk, N):
    _check_gateup(T, K, E, topk, N, seed=T + K + E + N)


def test_gate_up_prefill_sampled(gpu_available):
    rng = np.random.default_rng(8)
    rows = np.unique(rng.integers(0, 2048 * 8, 48))
    _check_gateup(2048, 2048, 16, 8, 128, seed=5, rows=rows)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_gate_up_scales_far_apart(gpu_available, T):
    _check_gateup(T, 1024, 4, 2, 128, seed=90 + T, spread=6, wide=9)


@pytest.mark.parametrize("T", [1, 5, 90, 400])
def test_gate_up_unused_and_crowded_experts(gpu_available, T):
    r = _check_gateup(T, 256, 6, 2, 192, seed=70 + T, bias=[0, -40, 9, 0, -40, 3])
    assert (np.diff(r["expert_off"]) == 0).sum() >= 2


def test_gate_up_non_finite_activations(gpu_available):
    """A NaN or infinity makes its token's outputs NaN and leaves the others as they were."""
    T, K, E, topk, N = 5, 256, 4, 2, 64
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    codes, scales = map(u8, _weights(rng, E, N, K, 2))
    r = _gpu_routing(_routing(T, E, topk, 3))
    print("gate_up with NaN and infinite activations", flush=True)
    gu0, _ = i8h.moe_gateup_mxfp4_grouped(x, codes, scales, topk, r["expert_off"], r["sorted_pairs"])
    x[1, 70], x[3, 5] = float("nan"), float("-inf")
    gu, act = i8h.moe_gateup_mxfp4_grouped(x, codes, scales, topk, r["expert_off"], r["sorted_pairs"])
    t = r["sorted_pairs"].long() // topk
    bad = (t == 1) | (t == 3)
    assert torch.isnan(gu[bad]).all() and torch.isnan(act[bad]).all()
    assert torch.equal(gu[~bad], gu0[~bad])


def _check_down(T, I, E, topk, H, seed, dtype, bias=None, tokens=None):
    rng = np.random.default_rng(seed)
    r = _routing(T, E, topk, seed, bias)
    P = T * topk
    a = rng.standard_normal((P, I)).clip(-3, 3) * 2
    a.reshape(P, -1, 32)[:, :, 0] = 4.5
    act = torch.from_numpy(a.astype(np.float32)).to(dtype)
    codes, scales = _weights(rng, E, H, I, 2)
    gr = _gpu_routing(r)
    print(f"down T={T} I={I} E={E} topk={topk} H={H} {dtype}", flush=True)
    out = i8h.moe_down_mxfp4_combine(act.cuda(), u8(codes), u8(scales), gr)
    torch.cuda.synchronize()
    qc, qs = mxfp4.quantize(values(act))
    pos = np.asarray(r["pair_pos"]).reshape(T, topk)
    tk = np.arange(T) if tokens is None else tokens
    need = np.unique(pos[tk])
    y, mag = mxfp4.grouped(mxfp4.dequantize(qc, qs), codes, scales, r["expert_off"], rows=need)
    assert mag.max() < 2.0 ** 24 * _units(qs, scales)        # y is exact in float32
    back = np.searchsorted(need, pos[tk])
    w = gr["topk_w"].cpu().numpy()[tk]
    ref, m = mxfp4.combine(y, w, back.reshape(-1))
    got = out.cpu().numpy().astype(np.float64)[tk]
    assert np.all(np.abs(got - ref) <= (topk + 1) * 2.0 ** -24 * m)


DOWN = [
    (1, 32, 1, 1, 32), (1, 768, 128, 8, 2048), (2, 96, 8, 2, 64), (3, 160, 5, 3, 96), (8, 704, 16, 8, 160),
    (9, 768, 60, 4, 352), (16, 416, 3, 1, 1056), (33, 1024, 2, 1, 128), (65, 256, 1, 1, 2048), (128, 768, 128, 8, 256),
    (200, 1056, 1, 1, 32), (300, 64, 3, 2, 576), (700, 32, 2, 2, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,I,E,topk,H", DOWN)
def test_down(gpu_available, T, I, E, topk, H, dtype):
    _check_down(T, I, E, topk, H, seed=T + I + E + H, dtype=dtype)


def test_down_prefill_sampled(gpu_available):
    _check_down(1999, 768, 16, 8, 256, seed=6, dtype=torch.bfloat16, tokens=np.arange(0, 1999, 97))


@pytest.mark.parametrize("T", [1, 5, 90, 400])
def test_down_unused_and_crowded_experts(gpu_available, T):
    _check_down(T, 288, 6, 2, 96, seed=50 + T, dtype=torch.float32, bias=[0, -40, 9, 0, -40, 3])


def test_zero_tokens_are_a_no_op(gpu_available):
    codes, scales = torch.zeros((4, 64, 128), dtype=torch.uint8, device="cuda"), \
        torch.zeros((4, 64, 8), dtype=torch.uint8, device="cuda")
    off, none = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    gu, act = i8h.moe_gateup_mxfp4_grouped(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), codes, scales, 2,
                                           off, none)
    assert gu.shape == (0, 64) and act.shape == (0, 32)
    r = {"topk_ids": torch.empty((0, 2), dtype=torch.int32, device="cuda"), "topk_w": torch.empty((0, 2), device="cuda"),
         "expert_off": off, "pair_pos": none}
    assert i8h.moe_down_mxfp4_combine(torch.empty((0, 256), device="cuda"), codes, scales, r).shape == (0, 64)


def test_rows_around_the_outputs_are_left_alone(gpu_available):
    """Outputs carved out of larger buffers: nothing before or behind them is written."""
    T, K, E, topk, N, H = 9, 256, 5, 2, 128, 96
    rng = np.random.default_rng(21)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    r = _gpu_routing(_routing(T, E, topk, 4))
    codes, scales = map(u8, _weights(rng, E, N, K, 2))
    dc, ds = map(u8, _weights(rng, E, H, N // 2, 2))
    P = T * topk
    big = {n: torch.full((rows + 2, width), 7.0, dtype=dt, device="cuda")
           for n, rows, width, dt in (("gu", P, N, torch.float32), ("act", P, N // 2, torch.float32),
                                      ("a16", P, N // 2, torch.bfloat16), ("out", T, H, torch.float32))}
    inner = {n: t[1:-1] for n, t in big.items()}
    print("outputs inside larger buffers", flush=True)
    for act in ("act", "a16"):
        i8h.moe_gateup_mxfp4_grouped(x, codes, scales, topk, r["expert_off"], r["sorted_pairs"], gate_up=inner["gu"],
                                     act=inner[act])
        i8h.moe_down_mxfp4_combine(inner[act], dc, ds, r, out=inner["out"])
    torch.cuda.synchronize()
    for n, t in big.items():
        assert (t[0] == 7).all() and (t[-1] == 7).all(), n


@pytest.mark.parametrize("T,K", [(4, 256), (40, 256), (600, 256), (20, 2304), (20, 8448)])
def test_gate_up_at_the_ends_of_float32(gpu_available, T, K):
    """Terms all alike, 2.25 or 9 times a power of two: their sums are exact down into the subnormals where the terms
    are multiples of 2^-149, and infinite past float32's range; below, they lose at most themselves."""
    N = 64
    r = {"expert_off": _i32([0, T]), "sorted_pairs": _i32(np.arange(T))}
    for sw in (0, 1, 20, 127, 250, 254):
        for ex in (-122, -30, -4, 0, 100, 125):
            for code, value in ((3, 1.5), (7, 6.0)):
                print(f"gate_up ends of float32 T={T} K={K} scale={sw} x=1.5*2^{ex} weight={value}", flush=True)
                x = torch.full((T, K), 1.5 * 2.0 ** ex).to(torch.bfloat16).cuda()
                gu, _ = i8h.moe_gateup_mxfp4_grouped(x, torch.full((1, N, K // 2), 17 * code, dtype=torch.uint8, device="cuda"),
                                                     torch.full((1, N, K // 32), sw, dtype=torch.uint8, device="cuda"), 1,
                                                     r["expert_off"], r["sorted_pairs"], act=False)
                term = 1.5 * value * 2.0 ** (ex + sw - 127)
                got = values(gu)
                if term * K >= 2.0 ** 128:
                    assert np.isinf(got).all() and (got > 0).all()
                elif term >= 2.0 ** -147:                # 2.25 and 9 are whole multiples of a quarter
                    assert (got == term * K).all()
                else:
                    assert ((got >= 0) & (got <= term * K)).all()

"""GPU parity: lora_add and linear_i8f16_lora against the oracle.

Bounds (float32 sums of exact products, 2^-23 a term): the adapters' part as
oracle/lora.py gives it, the linear's K 2^-23 sum |terms|, 2^-23 of the values
joined, and half a step of the output's type (bf16: 2^-8).
"""

import math

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import dense, lora

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def adapters(L, R, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn((L, R, K), generator=g) / math.sqrt(K)).to(BF16).cuda()
    b = (torch.randn((L, N, R), generator=g) / math.sqrt(R)).to(BF16).cuda()
    s = (0.25 + torch.rand((L,), generator=g)).cuda()
    return a, b, s


def rows_of(T, L, kind, seed):
    """The rows' adapters: every row another (none among them), runs of requests, one for all, none at all."""
    g = torch.Generator().manual_seed(seed)
    if kind == "mixed":
        ad = torch.randint(-1, L, (T,), generator=g)
    elif kind == "runs":
        ad = torch.randint(-1, L, (T,), generator=g)[torch.sort(torch.randint(0, max(1, T // 20) + 1, (T,), generator=g))[0].clamp(max=T - 1)]
    elif kind == "one":
        ad = torch.full((T,), L - 1)
    else:
        ad = torch.tensor([-1, L, -(1 << 31), (1 << 31) - 1])[torch.arange(T) % 4]
    return ad.int().cuda()


def problem(T, K, N, R, L, kind, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    x = torch.randn((T, K), generator=g).to(BF16).cuda()
    base = torch.randn((T, N), generator=g).to(dtype).cuda()
    return (base, x) + adapters(L, R, K, N, seed) + (rows_of(T, L, kind, seed),)


def check_add(out, base, x, a, b, s, ad):
    d, lim = lora.delta(f64(x), f64(a), f64(b), ad.cpu().numpy(), f64(s))
    ref = f64(base) + d
    lim = lim + 2.0 ** -23 * (np.abs(f64(base)) + np.abs(d))
    if base.dtype is BF16:
        lim = lim + 2.0 ** -8 * (np.abs(ref) + lim)
    got = f64(out)
    assert np.all(np.abs(got - ref) <= lim), np.max(np.abs(got - ref) / np.maximum(lim, 1e-30))
    none = (ad.cpu() < 0) | (ad.cpu() >= a.shape[0])
    assert torch.equal(out.cpu()[none], base.cpu()[none])


CASES = [(1, 64, 16, 8, 1, "one"), (1, 2048, 512, 16, 4, "one"), (3, 8, 1, 8, 2, "mixed"), (7, 136, 60, 16, 5, "mixed"),
         (16, 256, 100, 24, 3, "runs"), (17, 1000, 33, 40, 4, "mixed"), (33, 512, 60, 8, 8, "mixed"),
         (64, 384, 256, 16, 48, "mixed"), (65, 128, 1030, 64, 2, "runs"), (100, 264, 130, 72, 3, "runs"),
         (19, 640, 257, 136, 2, "mixed"), (9, 320, 64, 256, 3, "mixed"), (130, 1032, 96, 32, 6, "runs"),
         (40, 128, 48, 16, 3, "none"), (16, 2304, 300, 48, 16, "mixed"), (257, 72, 20, 16, 1, "one")]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,N,R,L,kind", CASES)
def test_add(gpu_available, T, K, N, R, L, kind, dtype):
    print(f"lora_add T={T} K={K} N={N} R={R} L={L} {kind} {dtype}", flush=True)
    base, x, a, b, s, ad = problem(T, K, N, R, L, kind, dtype)
    out = i8h.lora_add(base, x, a, b, ad, s)
    check_add(out, base, x, a, b, s, ad)
    kept = base.clone()
    assert i8h.lora_add(base, x, a, b, ad, s, out=base) is base          # in place
    assert torch.equal(base, out) and not torch.equal(kept, out) or kind == "none" or bool((ad < 0).all())


@pytest.mark.parametrize("T,R,kind", [(1500, 16, "runs"), (1100, 64, "mixed"), (2049, 32, "one"), (1200, 8, "none")])
def test_add_many_rows(gpu_available, T, R, kind):
    """Past the rows that get a workgroup an adapter."""
    base, x, a, b, s, ad = problem(T, 256, 192, R, 20, kind, F32)
    check_add(i8h.lora_add(base, x, a, b, ad, s), base, x, a, b, s, ad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_slices_of_wider_matrices(gpu_available, dtype, shift):
    """base, x and out as column slices, at offsets that vector accesses fit and that they do not; what lies beside the
    slice stays as it was."""
    T, K, N = 21, 192, 76
    base, x, a, b, s, ad = problem(T, K, N, 16, 3, "mixed", dtype)
    wide = torch.full((T, 3 * N + 5), 7.0, dtype=dtype, device="cuda")
    wx = torch.full((T, 3 * K), 5.0, dtype=BF16, device="cuda")
    vb, vx = wide[:, N + shift:2 * N + shift], wx[:, K:2 * K]
    vb.copy_(base)
    vx.copy_(x)
    want = i8h.lora_add(base, x, a, b, ad, s)
    res = torch.full((T, 2 * N + 3), 9.0, dtype=dtype, device="cuda")
    vo = res[:, shift:N + shift]
    i8h.lora_add(vb, vx, a, b, ad, s, out=vo)
    assert torch.equal(vo, want) and bool((res[:, :shift] == 9).all()) and bool((res[:, N + shift:] == 9).all())
    i8h.lora_add(vb, vx, a, b, ad, s, out=vb)
    assert torch.equal(vb, want)
    assert bool((wide[:, :N + shift] == 7).all()) and bool((wide[:, 2 * N + shift:] == 7).all())


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_broken_adapters_stay_in_their_rows(gpu_available, value):
    """NaN and infinities in adapter 1, in its scale and in its rows' inputs reach no row of another adapter or of none."""
    T, K, N, R = 37, 256, 80, 40
    for dtype in (F32, BF16):
        base, x, a, b, s, ad = problem(T, K, N, R, 4, "mixed", dtype)
        want = i8h.lora_add(base, x, a, b, ad, s)
        for what in range(4):
            a2, b2, s2, x2 = a.clone(), b.clone(), s.clone(), x.clone()
            (a2[1] if what == 0 else b2[1] if what == 1 else s2[1:2] if what == 2 else x2[ad == 1]).fill_(value)
            if what == 3:
                x2[ad == 1] = value
            got = i8h.lora_add(base, x2, a2, b2, ad, s2)
            mine = ad == 1
            assert torch.equal(got[~mine], want[~mine])
            assert not bool(torch.isfinite(got[mine].float()).any())


@pytest.mark.parametrize("T", [5, 300, 1500])
def test_rows_without_an_adapter_keep_their_bits(gpu_available, T):
    """NaN payloads, signed zeros and subnormals of base pass through, beside rows that have an adapter."""
    K, N, R = 64, 300, 16
    for dtype, bits in ((F32, torch.int32), (BF16, torch.int16)):
        base, x, a, b, s, ad = problem(T, K, N, R, 3, "mixed", dtype)
        info = torch.iinfo(bits)
        base = torch.randint(info.min, info.max, (T, N), dtype=bits, device="cuda").view(dtype)
        base[:, 0] = -0.0
        out = i8h.lora_add(base, x, a, b, ad, s)
        none = ad < 0
        assert bool(none.any()) and torch.equal(out.view(bits)[none], base.view(bits)[none])


def test_inner_sums_are_not_rounded(gpu_available):
    """h = 1 + 2^-20 with B = 2^10 and a base of -2^10: what a product of bf16 inner sums would lose comes out whole."""
    T, K, N, R = 5, 8, 16, 8
    x = torch.ones((T, K), dtype=BF16, device="cuda")
    a = torch.zeros((1, R, K), dtype=BF16, device="cuda")
    a[0, 0, 0], a[0, 0, 1] = 1.0, 2.0 ** -20
    b = torch.zeros((1, N, R), dtype=BF16, device="cuda")
    b[0, :, 0] = 1024.0
    base = torch.full((T, N), -1024.0, device="cuda")
    out = i8h.lora_add(base, x, a, b, torch.zeros(T, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda"))
    assert bool((out == 2.0 ** -10).all())


def test_empty_batch(gpu_available):
    base, x, a, b, s, ad = problem(1, 64, 16, 8, 2, "one", F32)
    assert i8h.lora_add(base[:0], x[:0], a, b, ad[:0], s).shape == (0, 16)


LINEAR = [(1, 128, 16, 8, 1, "one"), (5, 256, 48, 16, 2, "mixed"), (16, 512, 64, 16, 3, "one"),
          (17, 384, 32, 24, 3, "mixed"), (33, 1024, 64, 64, 4, "runs"), (16, 2048, 256, 16, 5, "mixed"),
          (20, 2560, 48, 32, 2, "runs"), (128, 512, 128, 16, 8, "runs"), (130, 256, 144, 40, 4, "mixed"),
          (300, 384, 272, 16, 6, "runs"), (513, 128, 112, 8, 3, "mixed"), (70, 640, 336, 256, 2, "runs"),
          (64, 256, 64, 16, 2, "none")]


@pytest.mark.parametrize("T,K,N,R,L,kind", LINEAR)
def test_linear(gpu_available, T, K, N, R, L, kind):
    print(f"linear_i8f16_lora T={T} K={K} N={N} R={R} L={L} {kind}", flush=True)
    _, x, a, b, s, ad = problem(T, K, N, R, L, kind, F32)
    g = torch.Generator().manual_seed(N)
    codes = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda()
    scales = (torch.rand((N, K // 128), generator=g) * 1e-2).to(torch.float16).cuda()
    scales[0] = 0
    scales[1] = 2.0 ** -20                    # f16 subnormals
    y = i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s)
    xf, sf = f64(x), scales.double().cpu().numpy()
    q = codes.cpu().numpy()
    lin = dense.linear_i8_f16(xf, q, sf)
    d, lim = lora.delta(xf, f64(a), f64(b), ad.cpu().numpy(), f64(s))
    lim = lim + K * 2.0 ** -23 * dense.linear_i8_f16(np.abs(xf), np.abs(q.astype(np.int32)), sf) \
        + 2.0 ** -23 * (np.abs(lin) + np.abs(d))
    assert np.all(np.abs(f64(y) - lin - d) <= lim)
    out = torch.full_like(y, math.nan)
    assert i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s, out=out) is out and torch.equal(out, y)


def test_linear_broken_adapters_stay_in_their_rows(gpu_available):
    T, K, N = 40, 256, 96
    _, x, a, b, s, ad = problem(T, K, N, 24, 4, "mixed", F32)
    codes = torch.randint(-127, 128, (N, K)).to(torch.int8).cuda()
    scales = torch.full((N, K // 128), 1e-3, dtype=torch.float16, device="cuda")
    want = i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s)
    for value in (math.nan, math.inf):
        b2 = b.clone()
        b2[2] = value
        got = i8h.linear_i8f16_lora(x, codes, scales, a, b2, ad, s)
        mine = ad == 2
        assert torch.equal(got[~mine], want[~mine]) and not bool(torch.isfinite(got[mine]).any())


def test_refusals(gpu_available):
    base, x, a, b, s, ad = problem(6, 64, 16, 8, 2, "one", F32)
    for bad in ((base.t(), x, a, b, ad, s), (base, x[:5], a, b, ad, s), (base, x, a[:, :, :56], b, ad, s),
                (base, x, a, b[:1], ad, s), (base, x, a, b, ad[:5], s), (base, x, a, b, ad, s[:1]),
                (base, x[:, ::2], a, b, ad, s), (base[0], x, a, b, ad, s), (base.expand(6, 16)[:1].expand(6, 16), x, a, b, ad, s)):
        with pytest.raises(ValueError):
            i8h.lora_add(*bad)
    for bad in ((base.half(), x, a, b, ad, s), (base, x.float(), a, b, ad, s), (base, x, a.float(), b, ad, s),
                (base, x, a, b, ad.long(), s), (base, x, a, b, ad, s.double())):
        with pytest.raises(TypeError):
            i8h.lora_add(*bad)
    big = problem(300, 64, 16, 8, 2, "one", F32)
    with pytest.raises(ValueError):
        i8h.lora_add(*big[:4], big[5], big[4], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(i8h.I8HError):                                   # ranks are multiples of 8
        i8h.lora_add(base, x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), ad, s)
    wide = torch.zeros((6, 40), device="cuda")
    with pytest.raises(i8h.I8HError):                                   # out meets base in part
        i8h.lora_add(wide[:, :16], x, a, b, ad, s, out=wide[:, 8:24])


def test_linear_refusals(gpu_available):
    T, K, N = 6, 128, 32
    _, x, a, b, s, ad = problem(T, K, N, 8, 2, "one", F32)
    codes = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    scales = torch.zeros((N, 1), dtype=torch.float16, device="cuda")
    for bad in ((x[:, :64], codes, scales, a, b, ad, s), (x, codes[:, :64], scales, a, b, ad, s), (x, codes, scales[:16], a, b, ad, s),
                (x, codes.t(), scales, a, b, ad, s), (x, codes, scales, a[:, :, :64], b, ad, s), (x, codes, scales, a, b[:, :16], ad, s),
                (x, codes, scales, a, b, ad[:5], s), (x, codes, scales, a, b, ad, s[:1]), (x[0], codes, scales, a, b, ad, s)):
        with pytest.raises(ValueError):
            i8h.linear_i8f16_lora(*bad)
    for bad in ((x.float(), codes, scales, a, b, ad, s), (x, codes.int(), scales, a, b, ad, s),
                (x, codes, scales.bfloat16(), a, b, ad, s), (x, codes, scales, a, b, ad.long(), s)):
        with pytest.raises(TypeError):
            i8h.linear_i8f16_lora(*bad)
    with pytest.raises(ValueError):
        i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(i8h.I8HError):                                   # columns are multiples of 16
        i8h.linear_i8f16_lora(x, codes[:24], scales[:24], a, b[:, :24].contiguous(), ad, s)
    assert i8h.linear_i8f16_lora(x[:0], codes, scales, a, b, ad[:0], s).shape == (0, N)

"""GPU parity of the adapters' kernels in each of their forms: one launch, 16
and 32 rows of lora_add, each tile of linear_i8f16_lora. Bounds as in
test_gpu_lora.py."""

import math

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import lora
from tests.test_gpu_batch_sizes import _check_linear, _linear
from tests.test_gpu_lora import BF16, F32, f64, problem

pytestmark = pytest.mark.gpu

# lora_add in one launch, 16 rows a workgroup, 32 rows a workgroup (1280 and 1290 of them)
ADD = [(5, 300), (300, 304), (8191, 1104)]
# linear_i8f16_lora's tiles: 16 x 16, 32 x 32, 64 x 128, 128 x 128
TILES = [(40, 48), (520, 272), (1030, 528), (2100, 1040)]


# --------------------------------------------------------------------------------------------------- infinities in B

def _formula(base, x, a, b, s, ad):
    """base + scale B (A x) in float64, for values small enough that only an operand's infinity gives one."""
    with np.errstate(invalid="ignore"):
        d, _ = lora.delta(f64(x), f64(a), f64(b), ad.cpu().numpy(), f64(s))
        return f64(base) + d


def _same_kind(got, ref, base, ad, L):
    g = f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    inf = np.isinf(ref)
    assert inf.any() and np.isnan(ref).any() and np.array_equal(np.isinf(g), inf) and np.array_equal(g[inf], ref[inf])


def _infinities(T, N, K, R, L):
    """Infinities and NaN in B at a few columns, beside inner sums that one bf16 holds, that take three, and that are 0."""
    base, x, a, b, s, ad = problem(T, K, N, R, L, "mixed", F32)
    a[:, 0] = 0
    a[:, 0, 1] = 1.0                       # h = x[1] scale, of few bits
    a[:, 1] = 0                            # h = 0
    s[:] = 0.5
    for l in range(L):
        b[l, 3, 0] = math.inf
        b[l, 7 % N, R - 1] = -math.inf     # h of full length
        b[l, 9 % N, 1] = math.inf          # times 0
        b[l, 17, 0], b[l, 17, 2] = math.inf, -math.inf
        b[l, 20, R - 2] = math.nan
        b[l, N - 1, 2 + l % 3] = math.inf
    return base, x, a, b, s, ad


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R", [8, 40])
@pytest.mark.parametrize("T,N", ADD)
def test_infinities_in_b(gpu_available, T, N, R, dtype):
    """An infinity times an inner sum is an infinity of its sign, NaN only where the sum is 0 or two of them meet, whatever
    the batch's size."""
    print(f"infinities in B T={T} N={N} R={R} {dtype}", flush=True)
    base, x, a, b, s, ad = _infinities(T, N, 72, R, 4)
    base = base.to(dtype)
    ref = _formula(base, x, a, b, s, ad)
    got = i8h.lora_add(base, x, a, b, ad, s)
    _same_kind(got, ref, base, ad, 4)
    # columns without one keep their bits
    b2 = torch.where(torch.isfinite(b.float()), b, torch.zeros_like(b))
    plain = i8h.lora_add(base, x, a, b2, ad, s)
    fine = torch.from_numpy(np.isfinite(ref)).cuda()
    assert torch.equal(got[fine], plain[fine])


@pytest.mark.parametrize("R", [8, 40, 168])
@pytest.mark.parametrize("T,N", TILES)
def test_infinities_in_b_of_the_linear(gpu_available, T, N, R):
    print(f"infinities in B, linear T={T} N={N} R={R}", flush=True)
    K = 256
    _, x, a, b, s, ad = _infinities(T, N, K, R, 4)
    codes, scales = _linear(K, N, T)
    zero = torch.zeros((T, N), device="cuda")
    ref = _formula(zero, x, a, b, s, ad)
    got = i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s)
    _same_kind(got, ref, zero, ad, 4)
    b2 = torch.where(torch.isfinite(b.float()), b, torch.zeros_like(b))
    plain = i8h.linear_i8f16_lora(x, codes, scales, a, b2, ad, s)
    fine = torch.from_numpy(np.isfinite(ref)).cuda()
    assert torch.equal(got[fine], plain[fine])
    _check_linear(plain, x, codes, scales, a, b2, s, ad)

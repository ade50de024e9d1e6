"""GPU parity of the adapters' and the scored routing's kernels in the forms
that only large batches take: 16 and 32 rows of lora_add, each tile of
linear_i8f16_lora, the scan of the routing's counts. Bounds as in
test_gpu_lora.py and test_gpu_scored.py; where sums are exact, equality."""

import math

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import lora, scored
from tests.test_gpu_batch_sizes import _check_linear, _linear
from tests.test_gpu_lora import BF16, F32, check_add, f64, problem
from tests.test_gpu_scored import bias_of, call, logits_of, rule

pytestmark = pytest.mark.gpu

# lora_add in one launch, 16 rows a workgroup, 32 rows a workgroup (1280 and 1290 of them)
ADD = [(5, 300), (300, 304), (8191, 1104)]
# linear_i8f16_lora's tiles: 16 x 16, 32 x 32, 64 x 128, 128 x 128
TILES = [(40, 48), (520, 272), (1030, 528), (2100, 1040)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,N,R,L,kind", [(8191, 72, 1104, 40, 6, "mixed"), (8192, 136, 1280, 16, 3, "runs"),
                                            (8225, 64, 1031, 72, 5, "runs"), (8191, 64, 1104, 256, 3, "mixed"),
                                            (16400, 40, 516, 8, 9, "mixed"), (33000, 64, 64, 232, 2, "runs")])
def test_add_by_32_rows(gpu_available, T, K, N, R, L, kind, dtype):
    """More than 1024 workgroups of 32 rows: whole and ragged ones, one step of R to eight, adapters mixed and in runs."""
    print(f"lora_add by 32 rows T={T} K={K} N={N} R={R} L={L} {kind} {dtype}", flush=True)
    base, x, a, b, s, ad = problem(T, K, N, R, L, kind, dtype)
    out = torch.full((T + 1, N), 3.0, dtype=dtype, device="cuda")
    i8h.lora_add(base, x, a, b, ad, s, out=out[:T])
    assert bool((out[T] == 3.0).all())
    check_add(out[:T], base, x, a, b, s, ad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [1, 4, 8])
def test_slices_by_32_rows(gpu_available, dtype, shift):
    """Column slices, on and off the vectors' alignment; what lies beside them stays."""
    T, K, N = 8200, 64, 1040
    base, x, a, b, s, ad = problem(T, K, N, 24, 4, "mixed", dtype)
    wide = torch.full((T, 2 * N + 24), 7.0, dtype=dtype, device="cuda")
    vb, vo = wide[:, shift:N + shift], wide[:, N + 16:2 * N + 16]
    vb.copy_(base)
    print(f"slices by 32 rows shift={shift} {dtype}", flush=True)
    i8h.lora_add(vb, x, a, b, ad, s, out=vo)
    check_add(vo, base, x, a, b, s, ad)
    assert torch.equal(vb, base) and bool((wide[:, N + shift:N + 16] == 7).all()) and bool((wide[:, 2 * N + 16:] == 7).all())
    want = vo.clone()
    i8h.lora_add(vb, x, a, b, ad, s, out=vb)
    assert torch.equal(vb, want) and torch.equal(vo, want)


# ------------------------------------------------------------------------------------- inner sums of 24 significant bits

def _whole_sums(T, N, K):
    """Inner sums 1 + 2^-12 + 2^-23, 1 and 1 + 2^-12, times a power of two a row, in columns 0, 33 and 130 of R. Even
    columns of the output are the first less the second times 2^10, odd ones the first less the third: every sum on the
    way is exact in float32, in any order."""
    R = 136
    g = torch.Generator().manual_seed(T)
    up = torch.randint(-3, 4, (T,), generator=g).float()
    x = torch.exp2(up)[:, None].expand(T, K).to(BF16).cuda()
    a = torch.zeros((2, R, K), dtype=BF16, device="cuda")
    a[1, [0, 33, 130], 3] = 1.0
    a[1, [0, 130], K // 2] = 2.0 ** -12
    a[1, 0, K - 1] = 2.0 ** -23
    b = torch.zeros((2, N, R), dtype=BF16, device="cuda")
    b[1, :, 0] = 1024.0
    b[1, 0::2, 33] = -1024.0
    b[1, 1::2, 130] = -1024.0
    ad = torch.randint(-1, 2, (T,), generator=g).int().cuda()
    want = torch.where(torch.arange(N) % 2 == 0, 0.25 + 2.0 ** -13, 2.0 ** -13)[None] * torch.exp2(up)[:, None]
    return x, a, b, ad, torch.tensor([1.0, 1.0], device="cuda"), torch.where((ad == 1).cpu()[:, None], want, 0.0 * want).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N", ADD)
def test_inner_sums_are_whole_in_every_add(gpu_available, T, N, dtype):
    print(f"whole inner sums T={T} N={N} {dtype}", flush=True)
    x, a, b, ad, s, want = _whole_sums(T, N, 520)
    out = i8h.lora_add(torch.zeros((T, N), dtype=dtype, device="cuda"), x, a, b, ad, s)
    assert torch.equal(out, want.to(dtype))
    # and of rank 8: five rows take one launch
    keep = [0, 33, 130, 1, 2, 3, 4, 5]
    out = i8h.lora_add(torch.zeros((T, N), dtype=dtype, device="cuda"), x, a[:, keep].contiguous(), b[:, :, keep].contiguous(),
                       ad, s)
    assert torch.equal(out, want.to(dtype))


@pytest.mark.parametrize("T,N", TILES)
def test_inner_sums_are_whole_in_every_tile(gpu_available, T, N):
    print(f"whole inner sums, linear T={T} N={N}", flush=True)
    K = 640
    x, a, b, ad, s, want = _whole_sums(T, N, K)
    codes = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    scales = torch.ones((N, K // 128), dtype=torch.float16, device="cuda")
    assert torch.equal(i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s), want)


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


# ----------------------------------------------------------------------------------------------- the scan of the counts

@pytest.mark.parametrize("T,E,k,groups,keep,top", [(4200, 60, 32, 1, 1, 1), (17000, 16, 3, 4, 2, 2), (16500, 160, 6, 8, 3, 1),
                                                   (16385, 384, 8, 6, 3, 2), (9000, 1000, 20, 4, 2, 2), (16400, 1024, 1, 1, 1, 1),
                                                   (70001, 64, 4, 1, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_more_chunks_than_one_scatter_adds_up(gpu_available, T, E, k, groups, keep, top, score):
    """More than 256 chunks: the permutation whole, against torch's stable sort; the choice against the oracle in a sample."""
    print(f"scored scan T={T} E={E} k={k} {score}", flush=True)
    l = logits_of(T, E, T, mask=0.05)
    r = rule(score, bias_of(E, 2), groups, keep, top, True, 2.5)
    got = call(l, k, r)
    flat = got["topk_ids"].flatten().long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(order.int(), got["sorted_pairs"])
    assert torch.equal(got["pair_pos"][order], torch.arange(T * k, dtype=torch.int32, device="cuda"))
    assert torch.equal(got["expert_off"], torch.searchsorted(flat[order].contiguous(), torch.arange(E + 1, device="cuda")).int())
    rows = torch.cat([torch.arange(0, T, 211), torch.tensor([T - 1])]).cuda()
    ref = scored.route(l[rows].cpu().numpy(), k, score, r["bias"], groups, keep, top, True, 2.5)
    assert np.array_equal(got["topk_ids"][rows].cpu().numpy(), ref["topk_ids"])
    # distances from the largest logit are below 40 here: (40 + 2 d) 2^-24
    w = got["topk_w"][rows].cpu().numpy()
    assert np.all(np.abs(w - ref["topk_w"]) <= 120 * 2.0 ** -24 * np.abs(ref["topk_w"]) + 2.0 ** -126)


# -------------------------------------------------------------------------------------- broken values in large batches

@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N", ADD[1:])
def test_broken_values_stay_in_their_rows(gpu_available, T, N, dtype, value):
    """NaN and infinities in an adapter, in its scale, in its rows' inputs, and in rows without one: the other rows' bits
    are those of the whole batch."""
    print(f"broken values T={T} N={N} {dtype} {value}", flush=True)
    base, x, a, b, s, ad = problem(T, 72, N, 40, 5, "mixed", dtype)
    want = i8h.lora_add(base, x, a, b, ad, s)
    mine, none = ad == 1, ad == -1
    for what in ("a", "b", "b here and there", "s", "x", "x of none"):
        a2, b2, s2, x2 = a.clone(), b.clone(), s.clone(), x.clone()
        if what == "a":
            a2[1] = value
        elif what == "b":
            b2[1] = value
        elif what == "b here and there":
            b2[1, ::17, 5] = value
        elif what == "s":
            s2[1] = value
        else:
            x2[mine if what == "x" else none] = value
        got = i8h.lora_add(base, x2, a2, b2, ad, s2)
        assert torch.equal(got[~mine], want[~mine]), what
        broken = torch.zeros(N, dtype=torch.bool, device="cuda")
        broken[::17] = what == "b here and there"
        if what in ("a", "b", "s", "x"):
            broken[:] = True
        assert not bool(torch.isfinite(got[mine][:, broken].float()).any()), what
        assert torch.equal(got[mine][:, ~broken], want[mine][:, ~broken]), what

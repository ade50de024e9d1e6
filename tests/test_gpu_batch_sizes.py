"""GPU parity of the scored routing and the adapters at sizes where tiles,
slices and offsets change: each tile of the linear, many rows of high rank,
rows and weights past 2^31 elements, logits off their vector alignment.
Bounds as in test_gpu_lora.py and test_gpu_scored.py."""

import math

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import dense, lora
from tests.test_gpu_lora import BF16, F32, check_add, f64, problem
from tests.test_gpu_scored import KEYS, bias_of, call, check, logits_of, rule

pytestmark = pytest.mark.gpu


def _linear(K, N, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda()
    return codes, (torch.rand((N, K // 128), generator=g) * 1e-2).to(torch.float16).cuda()


def _check_linear(y, x, codes, scales, a, b, s, ad):
    xf, q, sf = f64(x), codes.cpu().numpy(), scales.double().cpu().numpy()
    lin = dense.linear_i8_f16(xf, q, sf)
    d, lim = lora.delta(xf, f64(a), f64(b), ad.cpu().numpy(), f64(s))
    lim = lim + x.shape[1] * 2.0 ** -23 * dense.linear_i8_f16(np.abs(xf), np.abs(q.astype(np.int32)), sf) \
        + 2.0 ** -23 * (np.abs(lin) + np.abs(d))
    assert np.all(np.abs(f64(y) - lin - d) <= lim)


# 16 x 16 tiles, 32 x 32, 64 x 128, 128 x 128: each with ragged tokens, columns and groups of K
@pytest.mark.parametrize("T,N", [(500, 256), (520, 272), (1030, 528), (2100, 1040)])
@pytest.mark.parametrize("K,R,L,kind", [(128, 8, 3, "mixed"), (640, 136, 2, "runs"), (384, 16, 9, "mixed")])
def test_linear_tiles(gpu_available, T, N, K, R, L, kind):
    print(f"linear tiles T={T} N={N} K={K} R={R} L={L} {kind}", flush=True)
    _, x, a, b, s, ad = problem(T, K, N, R, L, kind, F32)
    codes, scales = _linear(K, N, T)
    y = torch.full((T + 1, N), 7.0, device="cuda")
    i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s, out=y[:T])
    assert bool((y[T] == 7.0).all())
    _check_linear(y[:T], x, codes, scales, a, b, s, ad)


@pytest.mark.parametrize("T,N", [(520, 272), (1030, 528), (2100, 1040)])
def test_linear_tiles_keep_broken_adapters_to_their_rows(gpu_available, T, N):
    K = 256
    _, x, a, b, s, ad = problem(T, K, N, 16, 4, "mixed", F32)
    codes, scales = _linear(K, N, 1)
    want = i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s)
    mine = ad == 2
    for what, value in ((0, math.nan), (1, math.inf), (2, math.nan)):
        v = [a.clone(), b.clone(), s.clone()]
        v[what][2] = value
        got = i8h.linear_i8f16_lora(x, codes, scales, v[0], v[1], ad, v[2])
        assert torch.equal(got[~mine], want[~mine]) and not bool(torch.isfinite(got[mine]).any())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,N,R,L,kind", [(66, 72, 700, 256, 3, "mixed"), (64, 64, 300, 64, 70, "mixed"),
                                            (64, 64, 300, 72, 9, "mixed"), (128, 264, 700, 32, 40, "mixed"), (129, 264, 700, 32, 40, "mixed"),
                                            (256, 520, 300, 16, 50, "mixed"), (257, 520, 300, 16, 50, "mixed"), (300, 520, 259, 200, 40, "mixed"),
                                            (1025, 40, 77, 24, 200, "mixed"), (5000, 136, 300, 72, 3, "runs")])
def test_add_sizes(gpu_available, T, K, N, R, L, kind, dtype):
    print(f"add sizes T={T} K={K} N={N} R={R} L={L} {kind} {dtype}", flush=True)
    base, x, a, b, s, ad = problem(T, K, N, R, L, kind, dtype)
    out = torch.full((T + 1, N), 3.0, dtype=dtype, device="cuda")
    i8h.lora_add(base, x, a, b, ad, s, out=out[:T])
    assert bool((out[T] == 3.0).all())
    check_add(out[:T], base, x, a, b, s, ad)


@pytest.mark.parametrize("T", [40, 300])
def test_rows_far_apart(gpu_available, T):
    """Rows 2^24 elements apart: with 300 of them offsets pass 2^31 elements and 2^32 bytes."""
    K, N, R, far = 64, 80, 16, 1 << 24
    base, x, a, b, s, ad = problem(T, K, N, R, 4, "mixed", BF16)
    want = i8h.lora_add(base, x, a, b, ad, s)
    print(f"rows far apart T={T}", flush=True)
    wide = torch.empty((T, far), dtype=BF16, device="cuda")
    vb, vx = wide[:, 128:128 + N], wide[:, 512:512 + K]
    vb.copy_(base)
    vx.copy_(x)
    got = torch.empty((T, far), dtype=BF16, device="cuda")[:, 8:8 + N]
    i8h.lora_add(vb, vx, a, b, ad, s, out=got)
    assert torch.equal(got, want)
    i8h.lora_add(vb, vx, a, b, ad, s, out=vb)
    assert torch.equal(vb, want) and torch.equal(vx, x)


@pytest.mark.parametrize("T", [9, 300])
def test_slices_side_by_side(gpu_available, T):
    """base, out and x as slices of one matrix, next to each other: nothing but out's columns changes."""
    N = K = 64
    base, x, a, b, s, ad = problem(T, K, N, 16, 3, "mixed", BF16)
    want = i8h.lora_add(base, x, a, b, ad, s)
    wide = torch.cat([base, torch.zeros_like(base), x], 1)
    for at in (0, 1):                                     # out after base; then before it, and x last
        wide = torch.roll(wide, at * N, 1)
        vb, vo, vx = (wide[:, N * i:N * i + N] for i in ((0, 1, 2) if at == 0 else (1, 2, 0)))
        vo.zero_()
        i8h.lora_add(vb, vx, a, b, ad, s, out=vo)
        assert torch.equal(vo, want) and torch.equal(vb, base) and torch.equal(vx, x)
        with pytest.raises(i8h.I8HError):
            i8h.lora_add(vb, vx, a, b, ad, s, out=wide[:, 8:8 + N])


def test_outputs_past_2_31_elements(gpu_available):
    """66000 rows of 32768 columns. Rows repeat a pattern, so the first ones say what the last are."""
    T, K, N, R, n = 66000, 64, 32768, 8, 2000
    base, x, a, b, s, ad = problem(n, K, N, R, 3, "mixed", BF16)
    rep = T // n
    print("lora_add past 2^31 elements", flush=True)
    big, bx, bad = base.repeat(rep, 1), x.repeat(rep, 1), ad.repeat(rep)
    i8h.lora_add(big, bx, a, b, bad, s, out=big)
    for i in (0, rep // 2, rep - 1):
        sl = slice(i * n, (i + 1) * n)
        check_add(big[sl][::97], base[::97], x[::97], a, b, s, ad[::97])


def test_weights_past_2_31_elements(gpu_available):
    """lora_b of 2^31 elements and codes of 2.4e9: the last columns, and the last adapter."""
    g = torch.Generator().manual_seed(5)
    T, K, N, R = 5, 64, 1 << 22, 256
    x = torch.randn((T, K), generator=g).to(BF16).cuda()
    a = (torch.randn((3, R, K), generator=g) / 8).to(BF16).cuda()
    s = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    ad = torch.tensor([2, 1, -1, 0, 2], dtype=torch.int32, device="cuda")
    base = torch.randn((T, N), device="cuda")
    b = torch.zeros((3, N, R), dtype=BF16, device="cuda")
    tail = (torch.randn((3, 50, R), generator=g) / 16).to(BF16).cuda()
    b[:, -50:] = tail
    print("lora_b past 2^31 elements", flush=True)
    out = i8h.lora_add(base, x, a, b, ad, s)
    assert torch.equal(out[:, :-50], base[:, :-50])
    check_add(out[:, -50:].contiguous(), base[:, -50:].contiguous(), x, a, tail, s, ad)
    del b, base, out
    T, K, N, R = 21, 2304, (1 << 20) + 16, 8
    _, x, a, _, s, ad = problem(T, K, 16, R, 3, "mixed", F32)
    codes = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    scales = torch.zeros((N, K // 128), dtype=torch.float16, device="cuda")
    b = torch.zeros((3, N, R), dtype=BF16, device="cuda")
    tail_c, tail_s = _linear(K, 48, 3)
    tail_b = torch.randn((3, 48, R), generator=g).to(BF16).cuda()
    codes[-48:], scales[-48:], b[:, -48:] = tail_c, tail_s, tail_b
    print("codes past 2^31 elements", flush=True)
    y = i8h.linear_i8f16_lora(x, codes, scales, a, b, ad, s)
    assert bool((y[:, :-48] == 0).all())
    _check_linear(y[:, -48:].contiguous(), x, tail_c, tail_s, a, tail_b, s, ad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k,groups,keep", [(3, 64, 4, 1, 1), (30, 256, 8, 8, 4), (200, 256, 8, 8, 4), (65, 60, 4, 3, 2),
                                               (9, 1024, 8, 1, 1)])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_logits_off_their_alignment(gpu_available, T, E, k, groups, keep, shift, dtype):
    lg = logits_of(T, E, T + shift, dtype)
    flat = torch.full((T * E + 8,), math.nan, dtype=dtype, device="cuda")
    off = flat[shift:shift + T * E].view(T, E)
    off.copy_(lg)
    r = rule("sigmoid", bias_of(E, 3), groups, keep, 2 if groups > 1 else 1)
    got = check(off, k, r), call(off, k, r), call(lg, k, r)
    assert all(torch.equal(got[1][key], got[2][key]) for key in KEYS + ("topk_w",))


def test_routing_past_2_31_logits(gpu_available):
    """2^25 + 3 tokens of 64 experts: rows repeat a pattern, so a small batch says what is chosen."""
    T, E, k, n = (1 << 25) + 3, 64, 2, 4096
    r = rule("sigmoid", bias_of(E, 1), 8, 3, 2, True, 2.0)
    part = logits_of(n, E, 9, BF16)
    want = call(part, k, r)
    print("routing past 2^31 logits", flush=True)
    lg = torch.empty((T, E), dtype=BF16, device="cuda")
    lg[:1 << 25].view(-1, n, E).copy_(part)
    lg[1 << 25:] = part[:3]
    got = call(lg, k, r)
    torch.cuda.synchronize()
    del lg
    for key in ("topk_ids", "topk_w"):
        assert bool((got[key][:1 << 25].view(-1, n, k) == want[key]).all()) and torch.equal(got[key][1 << 25:], want[key][:3])
    ids = got["topk_ids"].view(-1)
    count = torch.bincount(ids, minlength=E)
    assert torch.equal(got["expert_off"].long(), torch.cat([count.new_zeros(1), count.cumsum(0)]))
    sp = got["sorted_pairs"].long()
    assert bool((got["pair_pos"][sp] == torch.arange(T * k, device="cuda", dtype=torch.int32)).all())
    key = ids[sp].long() * (T * k) + sp               # sorted by expert, then by pair
    assert bool((key[1:] > key[:-1]).all())

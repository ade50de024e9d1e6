"""GPU parity of the MXFP4 products where their variants meet: rows of K longer
than a workgroup holds, batches on either side of each choice, routings that no
router gives, NaN scales, tensors past 2^31 elements, other streams. Tolerances
are those of test_gpu_mxfp4.py (exact where every partial sum is a float32
number, which each case asserts)."""

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import mxfp4
from tests.test_gpu_mxfp4 import (_act_bound, _check_down, _check_gateup, _gpu_routing, _i32, _routing, _units,
                                  _weights, u8, values)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------- lengths and choices

LONG = [
    (3, 4096, 4, 2, 64), (5, 6272, 3, 1, 64), (8, 14336, 2, 2, 64),         # one launch, rows in chunks of 2048
    (8, 16384, 2, 2, 64),                                                   # tokens' rows past LDS
    (20, 4096, 16, 2, 64), (64, 4096, 2, 2, 128), (20, 8192, 4, 1, 64),     # scales 16 blocks a load
    (20, 2304, 16, 2, 64), (64, 2304, 2, 2, 64), (21, 2176, 3, 1, 64), (70, 2688, 1, 1, 128),   # 4 blocks a load
    (20, 8448, 4, 2, 64), (70, 8448, 1, 1, 192), (200, 8832, 2, 1, 64),     # rows in stages
]


@pytest.mark.parametrize("T,K,E,topk,N", LONG)
def test_gate_up_long_rows(gpu_available, T, K, E, topk, N):
    _check_gateup(T, K, E, topk, N, seed=T + K + E + N)


# few tokens / many: T = 8, 9 and 32, 33.. pairs; passes of 32 and of 128 rows: 8 and more pairs an expert
BORDERS = [(8, 4, 8), (8, 5, 16), (8, 8, 8), (8, 9, 16), (9, 1, 4), (4, 8, 16), (3, 11, 32), (1, 32, 32), (2, 32, 32),
           (3, 22, 32), (16, 2, 4), (17, 2, 4), (32, 2, 4), (33, 2, 4), (34, 2, 4),
           (80, 2, 4), (81, 2, 4)]


@pytest.mark.parametrize("T,topk,E", BORDERS)
def test_gate_up_borders(gpu_available, T, topk, E):
    _check_gateup(T, 384, E, topk, 128, seed=T * topk + E)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,topk,E", BORDERS)
def test_down_borders(gpu_available, T, topk, E, dtype):
    _check_down(T, 352, E, topk, 96, seed=T * topk + E, dtype=dtype)


@pytest.mark.parametrize("T,I,E,topk,H", [
    (4, 2048, 8, 2, 64), (4, 2080, 8, 2, 64), (3, 1024, 32, 20, 32),       # the one-launch form's ends
    (20, 2080, 4, 2, 32), (150, 2080, 2, 1, 64), (150, 8736, 2, 1, 32),    # rows in stages
    (20, 2304, 4, 2, 32), (150, 2304, 2, 1, 64), (40, 4096, 8, 2, 64), (150, 4096, 2, 1, 32),
])
def test_down_long_rows(gpu_available, T, I, E, topk, H):
    _check_down(T, I, E, topk, H, seed=T + I + H, dtype=torch.float32)


# Passes of up to 128 rows (one expert) against 256 workgroups: a helper or more a pass, even runs over the workgroups
# left, whole remainders, no helper, none left, whole rounds and a few more.
PASSES = [2, 50, 128, 129, 135, 137, 160, 200, 255, 256, 257, 300, 520]


@pytest.mark.parametrize("N", [64, 704, 832])
@pytest.mark.parametrize("passes", PASSES)
def test_gate_up_deals(gpu_available, passes, N):
    T = 128 * passes - 61
    _check_gateup(T, 128, 1, 1, N, seed=passes + N, rows=np.unique(np.r_[np.arange(0, T, 61), T - 1]))


@pytest.mark.parametrize("H", [32, 352, 416])
@pytest.mark.parametrize("passes", PASSES)
def test_down_deals(gpu_available, passes, H):
    T = 128 * passes - 61
    _check_down(T, 64, 1, 1, H, seed=passes + H, dtype=torch.bfloat16, tokens=np.unique(np.r_[np.arange(0, T, 61), T - 1]))


@pytest.mark.parametrize("E,passes", [(16, 3), (128, 120), (200, 190), (256, 256), (300, 300), (700, 600)])
def test_deals_of_small_passes(gpu_available, E, passes):
    """Passes of a few rows (quantised by the product's own workgroups): one expert each."""
    T, topk = passes, 1
    rng = np.random.default_rng(passes)
    ids = rng.choice(E, passes, replace=False).reshape(T, topk)
    r = _routing_of(ids, E)
    K, N, H = 384, 704, 416
    x, a = _exact_values(rng, T, K), _exact_values(rng, T, 96)
    codes, scales = _weights(rng, E, N, K, 2)
    dc, ds = _weights(rng, E, H, 96, 2)
    print(f"deals of small passes E={E} passes={passes}", flush=True)
    gu, _ = i8h.moe_gateup_mxfp4_grouped(x.cuda(), u8(codes), u8(scales), topk, r["expert_off"], r["sorted_pairs"],
                                         act=False)
    out = i8h.moe_down_mxfp4_combine(a.cuda(), u8(dc), u8(ds), r)
    off, order = r["expert_off"].cpu().numpy(), r["sorted_pairs"].cpu().numpy()
    ref, mag = mxfp4.grouped(mxfp4.dequantize(*mxfp4.quantize(values(x)))[order], codes, scales, off)
    assert mag.max() < 2.0 ** 24 * 0.25 * 2.0 ** -7 and np.array_equal(values(gu), ref)
    y, mag = mxfp4.grouped(mxfp4.dequantize(*mxfp4.quantize(values(a))), dc, ds, off)
    ref, m = mxfp4.combine(y, r["topk_w"].cpu().numpy(), r["pair_pos"].cpu().numpy())
    assert np.all(np.abs(values(out) - ref) <= 2.0 ** -23 * m)


# ------------------------------------------------------------------------------------------------------ routings

def _routing_of(ids, E, seed=0):
    """The routing tensors of any expert choice [T, k], stably sorted by expert."""
    ids = np.asarray(ids)
    T, k = ids.shape
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    w = np.random.default_rng(seed).random((T, k)).astype(np.float32)
    return {"topk_ids": _i32(ids), "topk_w": torch.from_numpy(w).cuda(), "sorted_pairs": _i32(order),
            "pair_pos": _i32(pos), "expert_off": _i32(np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]))}


def _exact_values(rng, rows, K):
    x = rng.standard_normal((rows, K)).clip(-3, 3) * 2
    x.reshape(rows, -1, 32)[:, :, 0] = 4.5
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("T,k,ids", [
    (8, 8, "all"), (8, 3, "all"), (5, 8, "twice"), (2, 32, "all"), (40, 3, "all"), (40, 4, "twice"), (300, 2, "all"),
    (8, 8, "last"), (300, 2, "last"),
])
def test_an_expert_chosen_more_than_once(gpu_available, T, k, ids):
    """Every slot the same expert, or each token's slots in equal pairs: an expert's rows exceed the tokens."""
    E, K, N, H = 33, 256, 128, 64
    rng = np.random.default_rng(T * k)
    if ids == "twice":
        chosen = np.repeat(rng.integers(0, E, (T, k // 2)), 2, axis=1)
    else:
        chosen = np.full((T, k), 5 if ids == "all" else E - 1)
    r = _routing_of(chosen, E)
    x = _exact_values(rng, T, K)
    codes, scales = _weights(rng, E, N, K, 2)
    print(f"repeated experts T={T} k={k} {ids}", flush=True)
    gu, act = i8h.moe_gateup_mxfp4_grouped(x.cuda(), u8(codes), u8(scales), k, r["expert_off"], r["sorted_pairs"])
    qc, qs = mxfp4.quantize(values(x))
    xq = mxfp4.dequantize(qc, qs)[r["sorted_pairs"].cpu().numpy() // k]
    off = r["expert_off"].cpu().numpy()
    ref, mag = mxfp4.grouped(xq, codes, scales, off)
    assert mag.max() < 2.0 ** 24 * _units(qs, scales)
    got = values(gu)
    assert np.array_equal(got, ref)
    want, z = mxfp4.gelu_tanh_act(got)
    assert np.all(np.abs(values(act) - want) <= _act_bound(want, z, got[:, :N // 2], got[:, N // 2:]))

    a = _exact_values(rng, T * k, N // 2)
    codes, scales = _weights(rng, E, H, N // 2, 2)
    out = i8h.moe_down_mxfp4_combine(a.cuda(), u8(codes), u8(scales), r)
    qc, qs = mxfp4.quantize(values(a))
    y, mag = mxfp4.grouped(mxfp4.dequantize(qc, qs), codes, scales, off)
    assert mag.max() < 2.0 ** 24 * _units(qs, scales)
    ref, m = mxfp4.combine(y, r["topk_w"].cpu().numpy(), r["pair_pos"].cpu().numpy())
    assert np.all(np.abs(values(out) - ref) <= (k + 1) * 2.0 ** -24 * m)


@pytest.mark.parametrize("T", [4, 40, 400])
def test_gate_up_rows_behind_the_last_expert_are_left_alone(gpu_available, T):
    """expert_off that ends before the last pair (an expert's share of the pairs elsewhere)."""
    E, K, N, k = 6, 128, 64, 2
    r = _gpu_routing(_routing(T, E, k, T))
    off = r["expert_off"].clone()
    end = int(off[E - 2])
    off[E - 1:] = end                                       # the last two experts own nothing
    rng = np.random.default_rng(T)
    x = _exact_values(rng, T, K).cuda()
    codes, scales = map(u8, _weights(rng, E, N, K, 2))
    print(f"gate_up, rows behind the last T={T}", flush=True)
    full, _ = i8h.moe_gateup_mxfp4_grouped(x, codes, scales, k, r["expert_off"], r["sorted_pairs"])
    gu = torch.full((T * k, N), 7.0, device="cuda")
    act = torch.full((T * k, N // 2), 7.0, device="cuda")
    i8h.moe_gateup_mxfp4_grouped(x, codes, scales, k, off, r["sorted_pairs"], gate_up=gu, act=act)
    assert torch.equal(gu[:end], full[:end]) and (gu[end:] == 7).all() and (act[end:] == 7).all()


# ------------------------------------------------------------------------------------------------------ NaN scales

@pytest.mark.parametrize("T,K", [(5, 256), (40, 256), (500, 256), (20, 2304), (20, 4096), (20, 8448)])
def test_nan_weight_scales(gpu_available, T, K):
    """A NaN scale makes its output column NaN for its expert's rows, and nothing else."""
    E, k, N, H = 3, 1, 64, 64
    rng = np.random.default_rng(T + K)
    r = _gpu_routing(_routing(T, E, k, T))
    off = r["expert_off"].cpu().numpy()
    x = _exact_values(rng, T, K).cuda()
    codes, scales = _weights(rng, E, N, K, 2)
    print(f"NaN weight scales T={T} K={K}", flush=True)

    def gateup(s):
        return i8h.moe_gateup_mxfp4_grouped(x, u8(codes), u8(s), k, r["expert_off"], r["sorted_pairs"])[0].cpu().numpy()
    clean = gateup(scales)
    spots = [(0, 0, 0), (0, 33, K // 32 - 1), (1, 31, 5), (2, N - 1, K // 32 - 1), (2, 17, 3)]
    bad = scales.copy()
    nan = np.zeros((T * k, N), bool)
    for e, n, b in spots:
        bad[e, n, b] = 255
        nan[off[e]:off[e + 1], n] = True
    got = gateup(bad)
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], clean[~nan])

    a = _exact_values(rng, T * k, K).cuda()
    codes, scales = _weights(rng, E, H, K, 2)

    def down(s):
        return i8h.moe_down_mxfp4_combine(a, u8(codes), u8(s), r).cpu().numpy()
    clean = down(scales)
    bad = scales.copy()
    for e, n, b in spots:
        bad[e, n, b] = 255
    got = down(bad)
    nan = np.zeros((T, H), bool)
    ids = r["topk_ids"].cpu().numpy()[:, 0]
    for e, n, _ in spots:
        nan[ids == e, n] = True
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], clean[~nan])


@pytest.mark.parametrize("T", [3, 40, 300])
def test_down_non_finite_act_rows(gpu_available, T):
    """A NaN or infinite act value makes its token's outputs NaN and leaves the others as they were."""
    E, k, I, H = 4, 2, 96, 64
    rng = np.random.default_rng(T)
    r = _gpu_routing(_routing(T, E, k, T))
    act = _exact_values(rng, T * k, I).cuda()
    codes, scales = map(u8, _weights(rng, E, H, I, 2))
    print(f"down with NaN and infinite act rows T={T}", flush=True)
    clean = i8h.moe_down_mxfp4_combine(act, codes, scales, r)
    pos = r["pair_pos"].view(T, k)
    act[pos[1, 0], 95], act[pos[2, 1], 0] = float("nan"), float("inf")
    got = i8h.moe_down_mxfp4_combine(act, codes, scales, r)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[1] = bad[2] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


# ------------------------------------------------------------------------------------------------------ large sizes

def test_quantiser_past_2_32_elements(gpu_available):
    base = torch.randn((1 << 13, 2048), device="cuda").to(torch.bfloat16)
    n = 257
    x = torch.empty((n, 1 << 13, 2048), dtype=torch.bfloat16, device="cuda")
    x.copy_(base)
    x[-1] *= 4
    print("quantise past 2^32 elements", flush=True)
    assert x.numel() > 1 << 32
    c0, s0 = i8h.mxfp4_quantize(base)
    codes, scales = i8h.mxfp4_quantize(x)
    assert torch.equal(codes[0], c0) and torch.equal(codes[128], c0) and torch.equal(codes[-1], c0)
    assert torch.equal(scales[0], s0) and torch.equal(scales[-2], s0) and torch.equal(scales[-1], s0 + 2)
    i8h.mxfp4_dequantize(codes, scales, out=x)
    want = i8h.mxfp4_dequantize(c0, s0)
    assert torch.equal(x[0], want) and torch.equal(x[-2], want) and torch.equal(x[-1], want * 4)


def test_products_past_2_31_outputs(gpu_available):
    T, K, N = 70000, 128, 32768
    rng = np.random.default_rng(7)
    x = _exact_values(rng, T, K)
    codes, scales = _weights(rng, 1, N, K, 2)
    r = _routing_of(np.zeros((T, 1), np.int64), 1)
    rows = np.array([0, 1, 31, 32, 4095, 65535, 65536, T - 129, T - 128, T - 2, T - 1])
    print("gate_up and down past 2^31 outputs", flush=True)
    gu, act = i8h.moe_gateup_mxfp4_grouped(x.cuda(), u8(codes), u8(scales), 1, r["expert_off"], r["sorted_pairs"])
    assert gu.numel() > 1 << 31
    qc, qs = mxfp4.quantize(values(x))
    xq = mxfp4.dequantize(qc, qs)
    off = np.array([0, T])
    ref, mag = mxfp4.grouped(xq, codes, scales, off, rows=rows)
    assert mag.max() < 2.0 ** 24 * _units(qs, scales)
    got = values(gu[rows])
    assert np.array_equal(got, ref)
    want, z = mxfp4.gelu_tanh_act(got)
    assert np.all(np.abs(values(act[rows]) - want) <= _act_bound(want, z, got[:, :N // 2], got[:, N // 2:]))
    del gu, act
    out = i8h.moe_down_mxfp4_combine(x.cuda(), u8(codes), u8(scales), r)      # [T, 128] as act rows, H = 32768
    assert out.numel() > 1 << 31
    w = r["topk_w"].cpu().numpy()[rows].astype(np.float64)
    assert np.all(np.abs(values(out[rows]) - w * ref) <= 2.0 ** -23 * w * mag)


@pytest.mark.parametrize("T", [3, 40])
def test_weights_past_2_32_bytes(gpu_available, T):
    """Experts whose codes start past 2^32 bytes."""
    E, N, K, k = 520, 8192, 2048, 2
    gen = torch.Generator(device="cuda").manual_seed(T)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(120, 123, (E, N, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    assert codes.numel() > 1 << 32
    rng = np.random.default_rng(T)
    ids = np.stack([np.full(T, E - 1), np.full(T, 513)], 1)
    r = _routing_of(ids, E)
    x = _exact_values(rng, T, K)
    print(f"weights past 2^32 bytes T={T}", flush=True)
    gu, _ = i8h.moe_gateup_mxfp4_grouped(x.cuda(), codes, scales, k, r["expert_off"], r["sorted_pairs"], act=False)
    out = i8h.moe_down_mxfp4_combine(_pairs(x, k).cuda(), codes, scales, r)
    qc, qs = mxfp4.quantize(values(x))
    xq = mxfp4.dequantize(qc, qs)
    cols = np.concatenate([np.arange(64), np.arange(N // 2 - 32, N // 2 + 32), np.arange(N - 64, N)])
    y = {}
    for e, rows in ((513, slice(0, T)), (E - 1, slice(T, 2 * T))):
        w = mxfp4.dequantize(codes[e].cpu().numpy()[cols], scales[e].cpu().numpy()[cols])
        y[e] = xq @ w.T
        assert (np.abs(xq) @ np.abs(w).T).max() < 2.0 ** 24 * 0.25 * 2.0 ** (int(qs.min()) - 127 - 7)
        assert np.array_equal(values(gu[rows])[:, cols], y[e])
    w = r["topk_w"].cpu().numpy().astype(np.float64)
    # row p of the down call's act is token p // k: pair (t, j) lies at row pos, of token pos // k
    pos = r["pair_pos"].cpu().numpy().reshape(T, k)
    ref = w[:, :1] * y[E - 1][pos[:, 0] // k] + w[:, 1:] * y[513][pos[:, 1] // k]
    mag = np.abs(w[:, :1] * y[E - 1][pos[:, 0] // k]) + np.abs(w[:, 1:] * y[513][pos[:, 1] // k])
    assert np.all(np.abs(values(out)[:, cols] - ref) <= (k + 1) * 2.0 ** -24 * mag)


def _pairs(x, k):
    return x.repeat_interleave(k, 0)


# ---------------------------------------------------------------------------------------------------------- streams

@pytest.mark.parametrize("T", [4, 200])
def test_calls_at_once_on_two_streams(gpu_available, T):
    """Each call takes its stream and a workspace of its own: two run at once without meeting."""
    E, K, N, k, H = 8, 1024, 256, 2, 128
    rng = np.random.default_rng(T)
    sets = []
    for i in range(2):
        r = _gpu_routing(_routing(T, E, k, 10 * T + i))
        sets.append((_exact_values(rng, T, K).cuda(), *map(u8, _weights(rng, E, N, K, 2)),
                     *map(u8, _weights(rng, E, H, N // 2, 2)), r))

    def step(x, gc, gs, dc, ds, r):
        _, act = i8h.moe_gateup_mxfp4_grouped(x, gc, gs, k, r["expert_off"], r["sorted_pairs"], gate_up=False)
        out = i8h.moe_down_mxfp4_combine(act, dc, ds, r)
        return i8h.mxfp4_quantize(out) + (out,)
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    print(f"two streams T={T}", flush=True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_quantiser_of_one_row_past_2_32_elements(gpu_available):
    """A flat tensor: its last dimension does not fit 32 bits."""
    n = (1 << 32) + 96
    print("quantise a row past 2^32 elements", flush=True)
    base = torch.randn(1 << 16, device="cuda").to(torch.bfloat16)
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    x[:1 << 32].view(-1, 1 << 16).copy_(base)
    x[1 << 32:] = base[:96] * 4
    c0, s0 = i8h.mxfp4_quantize(base)
    codes, scales = i8h.mxfp4_quantize(x)
    assert codes.shape == (n // 2,) and scales.shape == (n // 32,)
    m = 1 << 31
    assert (codes[:m].view(-1, 1 << 15) == c0).all() and torch.equal(codes[m:], c0[:48])
    assert (scales[:m // 16].view(-1, 1 << 11) == s0).all() and torch.equal(scales[m // 16:], s0[:3] + 2)
    del x
    back = i8h.mxfp4_dequantize(codes, scales)
    want = i8h.mxfp4_dequantize(c0, s0)
    assert (back[:1 << 32].view(-1, 1 << 16) == want).all() and torch.equal(back[1 << 32:], want[:96] * 4)


# --------------------------------------------------------------------------------- each depth of the prefetch, reloads

# at most 8 pairs an expert and past the one-launch form: K to 768, to 1024, to 2048 take prefetches of their own
@pytest.mark.parametrize("T,K,E,topk,N", [(40, 768, 64, 2, 128), (40, 896, 64, 2, 64), (40, 1024, 64, 2, 128),
                                          (40, 1152, 64, 2, 64), (40, 1920, 64, 2, 64), (40, 2048, 64, 2, 128)])
def test_gate_up_small_passes_of_every_depth(gpu_available, T, K, E, topk, N):
    _check_gateup(T, K, E, topk, N, seed=T + K + E + N)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("I", [768, 800, 1024, 1056, 1536, 2016, 2048])
def test_down_small_passes_of_every_depth(gpu_available, I, dtype):
    _check_down(40, I, 64, 2, 96, seed=I, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("I", [768, 800, 1536, 2016, 2048, 2080, 2176, 2304, 6272, 8192, 8704])
def test_down_large_passes_of_every_kind(gpu_available, I, dtype):
    _check_down(90, I, 3, 2, 64, seed=I, dtype=dtype)


@pytest.mark.parametrize("T,k,K", [(8, 4, 2176), (8, 4, 4096), (1, 32, 4096), (5, 6, 6272)])
def test_one_launch_gate_up_takes_long_rows_for_more_than_sixteen_pairs(gpu_available, T, k, K):
    """Every slot the same expert: its weights, longer than a chunk, pass again for each sixteen pairs."""
    E, N = 33, 64
    r = _routing_of(np.full((T, k), 7), E)
    rng = np.random.default_rng(T * k + K)
    x = _exact_values(rng, T, K)
    codes, scales = _weights(rng, E, N, K, 2)
    print(f"one-launch gate_up, long rows T={T} k={k} K={K}", flush=True)
    gu, act = i8h.moe_gateup_mxfp4_grouped(x.cuda(), u8(codes), u8(scales), k, r["expert_off"], r["sorted_pairs"])
    _, a16 = i8h.moe_gateup_mxfp4_grouped(x.cuda(), u8(codes), u8(scales), k, r["expert_off"], r["sorted_pairs"],
                                          gate_up=False, act_dtype=torch.bfloat16)
    qc, qs = mxfp4.quantize(values(x))
    ref, mag = mxfp4.grouped(mxfp4.dequantize(qc, qs)[r["sorted_pairs"].cpu().numpy() // k], codes, scales,
                             r["expert_off"].cpu().numpy())
    assert mag.max() < 2.0 ** 24 * _units(qs, scales)
    got = values(gu)
    assert np.array_equal(got, ref)
    want, z = mxfp4.gelu_tanh_act(got)
    assert np.all(np.abs(values(act) - want) <= _act_bound(want, z, got[:, :N // 2], got[:, N // 2:]))
    assert torch.equal(a16, act.to(torch.bfloat16))

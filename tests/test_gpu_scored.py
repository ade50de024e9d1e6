"""GPU parity: moe_route_scored_permute against the oracle. Integer outputs are
equal, bit for bit. Weights: |w - ref| <= (40 + 2 d) 2^-24 |ref| + 2^-126 with
d the distance of the chosen logit from the row's largest (softmax; 0 for
sigmoid): float32 exponentials of a rounded argument (d 2^-24 each side of the
quotient, an ulp each), sums of up to 1024 positive terms by halves (10), two
quotients, a product; values below float32's smallest normal may be zero.
"""

import math

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import scored

pytestmark = pytest.mark.gpu

KEYS = ("topk_ids", "expert_off", "sorted_pairs", "pair_pos")


def rule(score="softmax", bias=None, groups=1, keep=1, top=1, renorm=True, scale=1.0):
    return dict(score=score, bias=bias, groups=groups, keep=keep, top=top, renorm=renorm, scale=scale)


def call(logits, k, r, **kw):
    bias = None if r["bias"] is None else torch.from_numpy(np.asarray(r["bias"], dtype=np.float32)).cuda()
    return i8h.moe_route_scored_permute(logits, k, score=r["score"], bias=bias, groups=r["groups"],
                                        topk_groups=r["keep"], group_top=r["top"], renormalize=r["renorm"],
                                        scale=r["scale"], **kw)


def check(logits, k, r, got=None):
    """logits: a float32 or bfloat16 tensor on the GPU."""
    got = call(logits, k, r) if got is None else got
    torch.cuda.synchronize()
    lg = logits.float().cpu().numpy().astype(np.float64)
    bias = None if r["bias"] is None else np.asarray(r["bias"], dtype=np.float32)
    ref = scored.route(lg, k, r["score"], bias, r["groups"], r["keep"], r["top"], r["renorm"], r["scale"])
    for key in KEYS:
        assert np.array_equal(got[key].cpu().numpy(), ref[key]), key
    w, want = got["topk_w"].cpu().numpy().astype(np.float64), ref["topk_w"]
    assert np.array_equal(np.isnan(w), np.isnan(want))
    with np.errstate(invalid="ignore"):
        d = np.zeros_like(want)
        if r["score"] == "softmax" and lg.size:
            d = np.nan_to_num(np.nanmax(lg, 1, keepdims=True) - np.take_along_axis(lg, ref["topk_ids"].astype(np.int64), 1),
                              posinf=0.0)
        ok = np.abs(w - want) <= (40 + 2 * d) * 2.0 ** -24 * np.abs(want) + 2.0 ** -126
    assert np.all(ok | np.isnan(want)), np.nanmax(np.abs(w - want) / np.abs(want))


def logits_of(T, E, seed, dtype=torch.float32, mask=0.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) * 2 + torch.randn((1, E), generator=g)
    if mask:
        l[torch.rand((T, E), generator=g) < mask] = -math.inf
        l[torch.rand((T,), generator=g) < 0.1] = -math.inf
    return l.to(dtype).cuda()


def bias_of(E, seed):
    return np.random.default_rng(seed).standard_normal(E).astype(np.float32) * 0.1


SHAPES = [(1, 1, 1, 1, 1), (1, 128, 8, 1, 1), (2, 60, 4, 1, 1), (4, 256, 8, 8, 4), (5, 160, 6, 8, 3), (3, 7, 7, 1, 1),
          (31, 64, 8, 4, 2), (33, 256, 8, 8, 4), (64, 65, 3, 5, 2), (77, 60, 4, 3, 2), (130, 1024, 32, 64, 9),
          (129, 512, 10, 16, 5), (200, 384, 9, 6, 6), (257, 12, 2, 6, 1), (513, 2, 1, 1, 1), (700, 256, 8, 32, 8),
          (1025, 128, 8, 1, 1), (300, 200, 25, 2, 1), (6, 1000, 20, 4, 2), (90, 300, 12, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,keep", SHAPES)
def test_shapes(gpu_available, T, E, k, groups, keep, score, dtype):
    print(f"scored T={T} E={E} k={k} groups={groups}/{keep} {score} {dtype}", flush=True)
    l = logits_of(T, E, T + E, dtype, mask=0.05 if T % 2 else 0.0)
    for seed, bias in enumerate((None, bias_of(E, E))):
        top = 2 if (seed + T) % 2 and E // groups >= 2 else 1
        check(l, k, rule(score, bias, groups, keep, top, renorm=bool((T + seed) % 3), scale=2.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(128, 1), (128, 8), (160, 8), (1024, 1), (40, 1)])
def test_choices_that_float32_cannot_tell_apart(gpu_available, E, groups, score):
    """Biases that bring every score + bias within a few 2^-25 of 1/2 (softmax: of 1/8): the order is that of float64."""
    T, k = 70, 6
    g = np.random.default_rng(E + groups)
    row = g.standard_normal(E).astype(np.float32)
    s = scored._score(row.astype(np.float64), score)
    bias = ((0.5 if score == "sigmoid" else 0.125) - s).astype(np.float32)
    l = np.repeat(row[None], T, 0)
    l[1::2] = np.nextafter(l[1::2], np.float32(9))      # half the rows a step away
    l[2::3, 0] += 1.0
    gaps = np.sort(s + bias.astype(np.float64))
    assert np.median(np.diff(gaps)) < 2.0 ** -28
    print(f"near E={E} groups={groups} {score}", flush=True)
    for top in (1, 2):
        check(torch.from_numpy(l).cuda(), k, rule(score, bias, groups, max(1, groups // 2), top))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_masks_and_special_values(gpu_available, score, bias):
    E, inf, nan = 48, math.inf, math.nan
    rows = np.zeros((16, E), dtype=np.float32)
    rows[1] = -inf
    rows[2] = -3.4028235e38                       # the type's lowest value
    rows[3, ::2] = -inf
    rows[4, 5] = nan
    rows[5] = nan
    rows[6, 7] = inf
    rows[7, 3:9] = -0.0
    rows[8] = np.arange(E) % 3
    rows[9, :46] = -inf
    rows[10] = np.linspace(-120, 120, E)          # scores that saturate
    rows[11] = 40 + np.arange(E) % 5              # 1 in float64 for a sigmoid
    rows[12] = -200
    rows[13, 20:] = nan
    rows[14] = np.where(np.arange(E) < 16, -inf, nan)
    b = np.tile(np.array([0.25, 0.0, -0.0, 0.25], dtype=np.float32), 12) if bias else None
    for T in (16, 64):
        l = torch.from_numpy(np.tile(rows, (T // 16, 1))).cuda()
        for groups, keep, top in ((1, 1, 1), (4, 2, 1), (4, 2, 2), (12, 3, 2), (3, 1, 2)):
            for renorm in (False, True):
                print(f"special T={T} {score} bias={bias} groups={groups}", flush=True)
                check(l, 8, rule(score, b, groups, keep, top, renorm))


def test_biases_that_are_not_numbers(gpu_available):
    E = 24
    b = np.zeros(E, dtype=np.float32)
    b[[1, 7]] = math.nan
    b[[2, 9]] = math.inf
    b[[3, 11]] = -math.inf
    l = logits_of(40, E, 3)
    for groups, keep, top in ((1, 1, 1), (4, 3, 1), (4, 3, 2)):
        check(l, E if groups == 1 else 18, rule("sigmoid", b, groups, keep, top))


def test_empty_batch(gpu_available):
    r = i8h.moe_route_scored_permute(torch.empty((0, 16), device="cuda"), 4)
    assert r["topk_ids"].shape == (0, 4)


def test_out_tensors_and_workspace_are_used(gpu_available):
    l = logits_of(300, 64, 1)
    first = call(l, 4, rule())
    again = call(l * 2, 4, rule(), out=first)
    assert all(again[key] is first[key] for key in first)
    check(l * 2, 4, rule(), again)
    with pytest.raises(ValueError):
        call(l, 4, rule(), out={"workspace": torch.empty(4, dtype=torch.uint8, device="cuda")})


@pytest.mark.parametrize("bad", [dict(topk=0), dict(topk=17), dict(groups=3), dict(groups=4, topk_groups=5),
                                 dict(groups=4, topk_groups=1, topk=5), dict(group_top=3), dict(score="tanh")])
def test_refusals(gpu_available, bad):
    kw = dict(topk=4, **{k: v for k, v in bad.items() if k != "topk"})
    kw["topk"] = bad.get("topk", 4)
    with pytest.raises((ValueError, i8h.I8HError)):
        i8h.moe_route_scored_permute(logits_of(3, 16, 0), **kw)


def test_bias_must_fit(gpu_available):
    l = logits_of(3, 16, 0)
    with pytest.raises(ValueError):
        i8h.moe_route_scored_permute(l, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        i8h.moe_route_scored_permute(l, 2, bias=torch.zeros(16, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        i8h.moe_route_scored_permute(l.t(), 2)


def test_long_batch(gpu_available):
    """Many chunks, against a torch form of the permutation and the oracle's choice on a sample of rows."""
    T, E, k = 40001, 256, 8
    l = logits_of(T, E, 9)
    r = rule("sigmoid", bias_of(E, 1), 8, 4, 2, True, 2.5)
    got = call(l, k, r)
    flat = got["topk_ids"].flatten().long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(order.int(), got["sorted_pairs"])
    assert torch.equal(got["pair_pos"][order], torch.arange(T * k, dtype=torch.int32, device="cuda"))
    assert torch.equal(got["expert_off"], torch.searchsorted(flat[order].contiguous(),
                                                             torch.arange(E + 1, device="cuda")).int())
    rows = torch.arange(0, T, 97, device="cuda")
    ref = scored.route(l[rows].cpu().numpy(), k, "sigmoid", r["bias"], 8, 4, 2, True, 2.5)
    assert np.array_equal(got["topk_ids"][rows].cpu().numpy(), ref["topk_ids"])
    assert np.abs(got["topk_w"][rows].cpu().numpy() / ref["topk_w"] - 1).max() <= 40 * 2.0 ** -24


SMALL = {"sigmoid": [[-60, -95], [-65, -90, -100], [-69, -120], [-86, -87, -88, -89], [-60, -100, -150, -700, -800, -3.4e38],
                     [-104, -105, -110, -300], [0, -95, -200], [-745, -746, -747], [-750, -1e30], [-60, -math.inf]],
         "softmax": [[0, -95], [-60, -95], [-60, -61, -95, -150], [-75, -80], [-300, -301, -700], [-800, -3.4e38],
                     [-60, -math.inf], [-86, -87, -88, -89]]}


@pytest.mark.parametrize("T", [20, 90])
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (True, 2.0 ** 90), (True, -2.0 ** 127), (False, 2.5),
                                          (False, 2.0 ** 120), (False, 2.0 ** -120)])
@pytest.mark.parametrize("by", ["bias", "groups", "logit"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_of_small_scores(gpu_available, score, by, renorm, scale, T):
    """Chosen scores far below one, and below float32's smallest normal value, keep the bound: each weight by itself, not
    as a part of the largest. Under softmax a bias (or, by two values, a group) keeps the largest logit, 0, out."""
    E, size = 24, 12
    rows = np.full((T, E), -math.inf, dtype=np.float32)
    bias = None
    for t in range(T):
        small = SMALL[score][t % len(SMALL[score])]
        rows[t, [(5 + t + 7 * j) % size for j in range(len(small))]] = small      # (7 and 12 share no factor)
        rows[t, size + t % size] = 0.0 if score == "softmax" else -math.inf
    if by == "bias":
        bias = np.where(np.arange(E) < size, 0.5, -0.5).astype(np.float32)
        bias[:size] += np.arange(size, dtype=np.float32) * np.float32(2.0 ** -6)
        r = rule(score, bias, 1, 1, 1, renorm, scale)
    elif by == "groups":
        bias = np.where(np.arange(E) < size, 1.0, -1.0).astype(np.float32)
        r = rule(score, bias, 2, 1, 2, renorm, scale)
    else:
        r = rule(score, None, 1, 1, 1, renorm, scale)
    l = torch.from_numpy(rows).cuda()
    got = call(l, 12, r)
    check(l, 12, r, got)
    w = got["topk_w"].cpu().numpy()
    assert np.all(w[np.take_along_axis(rows, got["topk_ids"].cpu().numpy().astype(np.int64), 1) == -math.inf] == 0)


def test_weights_of_spread_logits(gpu_available):
    """Sigmoid logits over -60 .. -130, where the scores leave float32's range one after the other."""
    g = torch.Generator().manual_seed(4)
    l = (-60 - 70 * torch.rand((700, 8), generator=g)).cuda()
    for renorm, scale in ((True, 1.0), (True, 2.0 ** 100), (False, 2.0 ** 100)):
        check(l, 8, rule("sigmoid", None, 1, 1, 1, renorm, scale))
        check(l, 4, rule("sigmoid", None, 4, 2, 2, renorm, scale))


@pytest.mark.parametrize("T", [9, 80])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scales_that_are_not_ordinary(gpu_available, score, T):
    """A scale of 0, an infinity or NaN meets each weight as its product in float64 does, rows masked whole among them."""
    l = logits_of(T, 40, T, mask=0.1)
    l[1] = -math.inf
    l[2, :38] = -math.inf
    for scale in (0.0, math.inf, -math.inf, math.nan, 3.4e38, 1e-45):
        for renorm in (True, False):
            r = rule(score, bias_of(40, 1), 4, 2, 1, renorm, scale)
            got = call(l, 6, r)
            with np.errstate(invalid="ignore", over="ignore"):
                one = scored.route(l.cpu().numpy(), 6, score, r["bias"], 4, 2, 1, renorm, 1.0)
                want = one["topk_w"] * float(np.float32(scale))
                w = got["topk_w"].cpu().numpy().astype(np.float64)
                assert np.array_equal(np.isnan(w), np.isnan(want)) and np.array_equal(got["topk_ids"].cpu().numpy(), one["topk_ids"])
                # distances from the largest logit are below 30 here: (40 + 2 d) 2^-24
                fine = (w == want) | np.isnan(want) | (np.abs(w - want) <= 100 * 2.0 ** -24 * np.abs(want) + 2.0 ** -126)
            assert fine.all(), (scale, renorm)

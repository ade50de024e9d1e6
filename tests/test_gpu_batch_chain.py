"""GPU: routing by scores and the low-rank adapters as a serving step uses
them: a projection with the requests' adapters, the router's logits with
theirs, experts by scores, the experts' products, adapters on their output,
then the drafted tokens checked; eagerly against the oracle of each new step,
on streams side by side, and captured in HIP graphs (two of which share their
workspaces)."""

import math

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import dense, draft, lora
from tests.test_gpu_graphs import ORDER, _capture, _check_replays
from tests.test_gpu_lora import adapters, check_add, f64
from tests.test_gpu_scored import check, rule

pytestmark = pytest.mark.gpu

E, K, N, TOPK, V, R, L = 16, 256, 128, 3, 300, 24, 5
I = N // 2
BF16 = torch.bfloat16


def _model(seed=0):
    g = torch.Generator().manual_seed(seed)
    w_up = torch.randn((E, N, K), generator=g) / K ** 0.5
    w_down = torch.randn((E, K, I), generator=g) / I ** 0.5
    return {"codes": torch.randint(-127, 128, (K, K), generator=g).to(torch.int8).cuda(),
            "scales": (torch.rand((K, K // 128), generator=g) * 1e-3).to(torch.float16).cuda(),
            "proj": adapters(L, R, K, K, seed + 1), "gate": (torch.randn((K, E), generator=g) / K ** 0.5).cuda(),
            "router": adapters(L, 8, K, E, seed + 2), "bias": 0.1 * torch.randn(E, generator=g).cuda(),
            "up": i8h.mxfp4_quantize(w_up.cuda()), "down": i8h.mxfp4_quantize(w_down.to(BF16).cuda()),
            "out": adapters(L, 2 * R, K, K, seed + 3), "head": (torch.randn((K, V), generator=g) / 4).cuda()}


RULE = rule("sigmoid", None, 4, 2, 2, True, 1.5)


def _step(m, x, ad):
    """Every intermediate of one step, in order."""
    y = i8h.linear_i8f16_lora(x, m["codes"], m["scales"], *m["proj"][:2], ad, m["proj"][2])
    h = y.to(BF16)
    plain = h.float() @ m["gate"]
    logits = i8h.lora_add(plain, h, *m["router"][:2], ad, m["router"][2])
    r = i8h.moe_route_scored_permute(logits, TOPK, score="sigmoid", bias=m["bias"], groups=4, topk_groups=2,
                                     group_top=2, scale=1.5)
    _, act = i8h.moe_gateup_mxfp4_grouped(h, *m["up"], TOPK, r["expert_off"], r["sorted_pairs"], gate_up=False,
                                          act_dtype=BF16)
    moe = i8h.moe_down_mxfp4_combine(act, *m["down"], r)
    out = i8h.lora_add(moe, h, *m["out"][:2], ad, m["out"][2])
    return y, h, plain, logits, r, moe, out


def _requests(B, D, seed):
    """Sequences of D + 1 positions, an adapter (or none) for each."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B * (D + 1), K), generator=g).to(BF16).cuda()
    return x, torch.randint(-1, L, (B,), generator=g).int().repeat_interleave(D + 1).cuda()


@pytest.mark.parametrize("B,D", [(1, 0), (1, 15), (3, 3), (20, 15), (70, 15)])
def test_serving_step(gpu_available, B, D):
    print(f"serving step B={B} D={D}", flush=True)
    m = _model()
    x, ad = _requests(B, D, B)
    y, h, plain, logits, r, moe, out = _step(m, x, ad)
    torch.cuda.synchronize()
    a, b, s = m["proj"]
    xf, q, sf = f64(x), m["codes"].cpu().numpy(), m["scales"].double().cpu().numpy()
    lin = dense.linear_i8_f16(xf, q, sf)
    d, lim = lora.delta(xf, f64(a), f64(b), ad.cpu().numpy(), f64(s))
    lim = lim + K * 2.0 ** -23 * dense.linear_i8_f16(np.abs(xf), np.abs(q.astype(np.int32)), sf) \
        + 2.0 ** -23 * (np.abs(lin) + np.abs(d))
    assert np.all(np.abs(f64(y) - lin - d) <= lim)
    check_add(logits, plain, h, *m["router"], ad)
    check(logits, TOPK, dict(RULE, bias=m["bias"].cpu().numpy()), got=r)
    check_add(out, moe, h, *m["out"], ad)
    if D > 0:
        g = torch.Generator().manual_seed(B)
        p = torch.softmax(out @ m["head"], -1).view(B, D + 1, V)
        drafted = p[:, :D].argmax(-1).int()
        u, un = torch.rand((B, D), generator=g).cuda(), torch.rand(B, generator=g).cuda()
        tokens, accepted = i8h.draft_verify(p, None, drafted, u, un)
        n = lambda t: t.cpu().numpy()  # noqa: E731
        want_t, want_n = draft.verify_batch(n(p).astype(np.float64), None, n(drafted), None, n(u), n(un))
        assert np.array_equal(n(accepted), want_n) and np.array_equal(n(tokens), want_t)


def test_requests_do_not_meet(gpu_available):
    """A request's results do not depend on which others share its batch: same rows, other neighbours, same bits (the
    sizes, and with them the kernels' forms, stay)."""
    m = _model()
    x, ad = _requests(6, 7, 3)
    one = _step(m, x, ad)
    x2, ad2 = _requests(6, 7, 4)
    x2[16:24], ad2[16:24] = x[16:24], ad[16:24]
    x2[:8] = math.nan
    two = _step(m, x2, ad2)
    for i in (0, 2, 3):
        assert torch.equal(one[i][16:24], two[i][16:24])
    for key in ("topk_ids", "topk_w"):
        assert torch.equal(one[4][key][16:24], two[4][key][16:24])


def test_two_streams(gpu_available):
    """Each call takes its stream and a workspace of its own: two run at once without meeting."""
    m = _model()
    sets = [_requests(20, 15, 1), _requests(70, 15, 2)]
    flat = lambda o: [o[0], o[3], o[5], o[6]] + [o[4][k] for k in ("topk_ids", "topk_w", "expert_off", "sorted_pairs", "pair_pos")]  # noqa: E731
    want = [[t.clone() for t in flat(_step(m, *s))] for s in sets]
    torch.cuda.synchronize()
    print("two streams", flush=True)
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for rep in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(flat(_step(m, *sets[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[i]))


def _step_fn(T, ws):
    """The new calls on fixed buffers, their workspaces carved by `ws(name, bytes)`."""
    m, lib = _model(3), i8h.lib()
    buf = {"x": torch.zeros((T, K), dtype=BF16, device="cuda"), "ad": torch.zeros(T, dtype=torch.int32, device="cuda")}
    o = {"y": torch.empty((T, K), device="cuda"), "logits": torch.empty((T, E), device="cuda"),
         "out": torch.empty((T, K), dtype=BF16, device="cuda")}
    w = {"proj": ws("proj", lib.lora_workspace_size(T, R)), "router": ws("router", lib.lora_workspace_size(T, 8)),
         "out": ws("out", lib.lora_workspace_size(T, 2 * R)),
         "route": ws("route", lib.moe_route_scored_workspace_size(T, E, TOPK))}
    route = {"topk_ids": torch.empty((T, TOPK), dtype=torch.int32, device="cuda"),
             "topk_w": torch.empty((T, TOPK), device="cuda"),
             "expert_off": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
             "sorted_pairs": torch.empty(T * TOPK, dtype=torch.int32, device="cuda"),
             "pair_pos": torch.empty(T * TOPK, dtype=torch.int32, device="cuda")}
    if w["route"] is not None:
        route["workspace"] = w["route"]

    def fn():
        i8h.linear_i8f16_lora(buf["x"], m["codes"], m["scales"], *m["proj"][:2], buf["ad"], m["proj"][2], out=o["y"],
                              workspace=w["proj"])
        o["logits"].copy_(buf["x"][:, :E])
        i8h.lora_add(o["logits"], buf["x"], *m["router"][:2], buf["ad"], m["router"][2], out=o["logits"],
                     workspace=w["router"])
        i8h.moe_route_scored_permute(o["logits"], TOPK, bias=m["bias"], groups=4, topk_groups=2, out=route)
        o["out"].copy_(o["y"])
        i8h.lora_add(o["out"], buf["x"], *m["out"][:2], buf["ad"], m["out"][2], out=o["out"], workspace=w["out"])
    names = ("topk_ids", "topk_w", "expert_off", "sorted_pairs", "pair_pos")
    return buf, fn, lambda: [o[k] for k in o] + [route[k] for k in names]


def _own(name, need):
    return torch.full((need,), 0xa5, dtype=torch.uint8, device="cuda") if need else None


def _input_sets(T, seed):
    g = torch.Generator().manual_seed(seed)
    return [[torch.randn((T, K), generator=g).to(BF16).cuda(), torch.randint(-1, L, (T,), generator=g).int().cuda()]
            for _ in range(2)]


@pytest.mark.parametrize("T", [1, 16, 80, 1200, 70000])
def test_captured_step(gpu_available, T):
    print(f"captured step T={T}", flush=True)
    buf, fn, outputs = _step_fn(T, _own)
    _check_replays(list(buf.values()), _input_sets(T, T), fn, outputs)


def test_two_graphs_share_workspaces(gpu_available):
    """Two captured steps of different sizes take the same bytes as workspaces; replayed in turn, with eager calls on
    those bytes between, each gives its own results."""
    pool = {}

    def shared(name, need):
        if name not in pool:
            pool[name] = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
        assert need <= pool[name].numel()
        return pool[name]
    print("two graphs, the same workspaces", flush=True)
    steps = []
    for T in (80, 1200):
        buf, fn, outputs = _step_fn(T, shared)
        sets, want = _input_sets(T, T), []
        for s in sets:
            for b, src in zip(buf.values(), s):
                b.copy_(src)
            fn()
            torch.cuda.synchronize()
            want.append([t.clone() for t in outputs()])
        steps.append((buf, sets, fn, outputs, want, _capture(fn)))
    for k in ORDER:
        for buf, sets, fn, outputs, want, graph in steps:
            for b, src in zip(buf.values(), sets[k]):
                b.copy_(src)
            graph.replay()
        torch.cuda.synchronize()
        for buf, sets, fn, outputs, want, graph in steps:
            assert all(torch.equal(a, w) for a, w in zip(outputs(), want[k]))
        steps[k][2]()
        for t in pool.values():
            t.fill_(0x5a)
        torch.cuda.synchronize()

"""GPU: the MXFP4 experts and the verification of drafted tokens as a serving
step uses them: quantised weights, router, gate_up, down, then the drafted
tokens checked against the target's distribution; eagerly against the oracle
of each step, and captured in HIP graphs (two of which share a workspace)."""

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import draft, mxfp4
from tests.test_gpu_graphs import ORDER, _capture, _check_replays
from tests.test_gpu_mxfp4 import _act_bound, values

pytestmark = pytest.mark.gpu

E, K, N, TOPK, V = 8, 256, 128, 2, 500
I = N // 2


def _model(seed=0):
    g = torch.Generator().manual_seed(seed)
    w_up = torch.randn((E, N, K), generator=g) / K ** 0.5
    w_down = torch.randn((E, K, I), generator=g) / I ** 0.5
    head = torch.randn((K, V), generator=g) / 4
    gate = torch.randn((K, E), generator=g) / K ** 0.5
    m = {"up": i8h.mxfp4_quantize(w_up.cuda()), "down": i8h.mxfp4_quantize(w_down.to(torch.bfloat16).cuda()),
         "head": head.cuda(), "gate": gate.cuda()}
    return m


def _layer(m, x, act_dtype, rotate=False, out=None):
    logits = x.float() @ m["gate"]
    if rotate:
        x = i8h.hadamard128_rotate(x)
    r = i8h.moe_route_permute(logits, TOPK)
    gu, act = i8h.moe_gateup_mxfp4_grouped(x, *m["up"], TOPK, r["expert_off"], r["sorted_pairs"], act_dtype=act_dtype)
    return r, x, gu, act, i8h.moe_down_mxfp4_combine(act, *m["down"], r)


@pytest.mark.parametrize("act_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("B,D", [(1, 3), (1, 15), (3, 15), (20, 15)])
def test_serving_step(gpu_available, B, D, act_dtype, rotate):
    """B sequences with D drafted tokens each: one verify batch of B (D + 1) tokens through the experts, then the
    tokens that stay. Each step is checked against its oracle on the step's own inputs."""
    T = B * (D + 1)
    m = _model()
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    print(f"serving step B={B} D={D} rotate={rotate} {act_dtype}", flush=True)
    r, xr, gu, act, out = _layer(m, x, act_dtype, rotate)
    p = torch.softmax(out @ m["head"], -1).view(B, D + 1, V)
    q = torch.softmax((out + 0.2 * torch.randn(out.shape, generator=g).cuda()) @ m["head"], -1).view(B, D + 1, V)
    q = q[:, :D].contiguous()
    drafted = q.argmax(-1).int()
    u, un = torch.rand((B, D), generator=g).cuda(), torch.rand(B, generator=g).cuda()
    tokens, accepted = i8h.draft_verify(p, q, drafted, u, un)
    greedy = i8h.draft_verify(p, None, drafted, u, un)
    torch.cuda.synchronize()

    off, sp = r["expert_off"].cpu().numpy(), r["sorted_pairs"].cpu().numpy()
    c, s = (t.cpu().numpy() for t in m["up"])
    xq = mxfp4.dequantize(*mxfp4.quantize(values(xr)))[sp // TOPK]
    ref, mag = mxfp4.grouped(xq, c, s, off)
    got = values(gu)
    assert np.all(np.abs(got - ref) <= K * 2.0 ** -23 * mag)
    want, z = mxfp4.gelu_tanh_act(got)
    lim = _act_bound(want, z, got[:, :I], got[:, I:])
    half = 2.0 ** -8 if act_dtype is torch.bfloat16 else 0.0
    assert np.all(np.abs(values(act) - want) <= lim + half * (np.abs(want) + lim) + 2.0 ** -134)
    c, s = (t.cpu().numpy() for t in m["down"])
    y, mag = mxfp4.grouped(mxfp4.dequantize(*mxfp4.quantize(values(act))), c, s, off)
    w, pos = r["topk_w"].cpu().numpy(), r["pair_pos"].cpu().numpy()
    ref, mo = mxfp4.combine(y, w, pos)
    y_err, _ = mxfp4.combine(I * 2.0 ** -23 * mag, w, pos)
    assert np.all(np.abs(values(out) - ref) <= (TOPK + 1) * 2.0 ** -24 * (mo + y_err) + y_err)
    n = lambda t: t.cpu().numpy()  # noqa: E731
    for draft_probs, (t, a) in ((n(q).astype(np.float64), (tokens, accepted)), (None, greedy)):
        want_t, want_n = draft.verify_batch(n(p).astype(np.float64), draft_probs, n(drafted), None, n(u), n(un))
        assert np.array_equal(n(a), want_n) and np.array_equal(n(t), want_t)


def _step_fn(T, B, D, ws):
    """A whole step on fixed buffers, its workspaces carved by `ws(name, bytes)`."""
    m = _model(3)
    lib = i8h.lib()
    buf = {"x": torch.zeros((T, K), dtype=torch.bfloat16, device="cuda"),
           "u": torch.zeros((B, D), device="cuda"), "un": torch.zeros(B, device="cuda")}
    drafted = (torch.arange(B * D, dtype=torch.int32, device="cuda") % V).view(B, D)
    o = {"act": torch.empty((T * TOPK, I), dtype=torch.bfloat16, device="cuda"), "out": torch.empty((T, K), device="cuda"),
         "codes": torch.empty((T, K // 2), dtype=torch.uint8, device="cuda"),
         "scales": torch.empty((T, K // 32), dtype=torch.uint8, device="cuda"),
         "back": torch.empty((T, K), device="cuda"), "p": torch.empty((B, D + 1, V), device="cuda"),
         "tokens": torch.empty((B, D + 1), dtype=torch.int32, device="cuda"),
         "accepted": torch.empty(B, dtype=torch.int32, device="cuda"), "logits": torch.empty((T, E), device="cuda")}
    w = {"up": ws("up", lib.moe_gateup_mxfp4_workspace_size(T, K, E, TOPK)),
         "down": ws("down", lib.moe_down_mxfp4_workspace_size(T, I, E, K, TOPK)),
         "draft": ws("draft", lib.draft_verify_workspace_size(B, V))}
    route = i8h.moe_route_permute(o["logits"].normal_(), TOPK)

    def fn():
        o["logits"].copy_(buf["x"][:, :E])
        r = i8h.moe_route_permute(o["logits"], TOPK, out=route)
        i8h.moe_gateup_mxfp4_grouped(buf["x"], *m["up"], TOPK, r["expert_off"], r["sorted_pairs"], gate_up=False,
                                     act=o["act"], act_dtype=torch.bfloat16, workspace=w["up"])
        i8h.moe_down_mxfp4_combine(o["act"], *m["down"], r, out=o["out"], workspace=w["down"])
        i8h.mxfp4_quantize(o["out"], codes=o["codes"], scales=o["scales"])
        i8h.mxfp4_dequantize(o["codes"], o["scales"], out=o["back"])
        o["p"].copy_(o["back"].abs().repeat(1, 2)[:, :V].reshape(B, D + 1, V))
        i8h.draft_verify(o["p"], None, drafted, buf["u"], buf["un"], tokens=o["tokens"], accepted=o["accepted"],
                         workspace=w["draft"])
    names = ("act", "out", "codes", "scales", "back", "tokens", "accepted")
    return buf, fn, lambda: [o[k] for k in names]


def _own(name, need):
    return torch.full((max(need, 1),), 0xa5, dtype=torch.uint8, device="cuda") if need else None


def _input_sets(T, B, D, seed):
    g = torch.Generator().manual_seed(seed)
    return [[torch.randn((T, K), generator=g).to(torch.bfloat16).cuda(), 0.05 * torch.rand((B, D), generator=g).cuda(),
             torch.rand(B, generator=g).cuda()] for _ in range(2)]


@pytest.mark.parametrize("B,D", [(1, 3), (2, 15), (20, 15)])
def test_captured_step(gpu_available, B, D):
    T = B * (D + 1)
    print(f"captured step B={B} D={D}", flush=True)
    buf, fn, outputs = _step_fn(T, B, D, _own)
    _check_replays(list(buf.values()), _input_sets(T, B, D, T), fn, outputs)


def test_two_graphs_share_a_workspace(gpu_available):
    """Two captured steps of different sizes take the same bytes as workspace; replayed in turn, with eager calls on
    those bytes between, each gives its own results."""
    pool = {}

    def shared(name, need):
        if name not in pool:
            pool[name] = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
        assert need <= pool[name].numel()
        return pool[name]
    print("two graphs, one workspace", flush=True)
    steps = []
    for B, D in ((2, 15), (20, 15)):
        buf, fn, outputs = _step_fn(B * (D + 1), B, D, shared)
        sets = _input_sets(B * (D + 1), B, D, B)
        want = []
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
        steps[k][2]()      # an eager call on the shared bytes
        for t in pool.values():
            t.fill_(0x5a)
        torch.cuda.synchronize()

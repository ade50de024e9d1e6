"""Routing by scores and low-rank adapters: cases, inputs, plain forms.

Three operators, each through the package's public call (`own` true) or in plain torch (`own` false):

  route       moe_route_scored_permute: experts by softmax or sigmoid scores, a bias for balance, groups, top-k,
              renormalised weights, and the expert-sorted permutation that the grouped products take
  lora        lora_add: low-rank adapters of many requests beside a shared projection's output
  linear      linear_i8f16_lora: the dense int8 linear with f16 scales and the requests' adapters in one product
"""

import math

import torch

own = False


# ---------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token of the layer whose experts the package multiplies: latency
        dict(name="route_decode", op="route", T=1, E=128, topk=8, score="softmax", bias=False, groups=1, keep=1, top=1,
             renorm=True, scale=1.0, dtype="f32", masked=False),
        # a verify batch, 8 sequences x (1 + 15 drafted), a router balanced by a bias
        dict(name="route_verify", op="route", T=128, E=128, topk=8, score="sigmoid", bias=True, groups=1, keep=1, top=1,
             renorm=True, scale=2.5, dtype="f32", masked=False),
        # an odd prefill chunk, bfloat16 logits, groups of 20 by their best expert, some experts switched off and some
        # rows of padding
        dict(name="route_groups", op="route", T=1999, E=160, topk=6, score="softmax", bias=False, groups=8, keep=3,
             top=1, renorm=False, scale=16.0, dtype="bf16", masked=True),
        # a long prefill chunk of a router with groups and a bias
        dict(name="route_prefill", op="route", T=16384, E=256, topk=8, score="sigmoid", bias=True, groups=8, keep=4,
             top=2, renorm=True, scale=2.5, dtype="f32", masked=False),
        # one decoded token with its request's adapter: latency
        dict(name="lora_decode", op="lora", T=1, requests=1, K=2048, N=2048, R=16, L=8, dtype="f32"),
        # a decode batch, a request a row, most with an adapter of their own
        dict(name="lora_requests", op="lora", T=64, requests=64, K=2048, N=4096, R=16, L=48, dtype="bf16"),
        # adapters beside the router's own small product
        dict(name="lora_router", op="lora", T=33, requests=33, K=2048, N=60, R=8, L=8, dtype="f32"),
        # a prefill chunk of five requests
        dict(name="lora_prefill", op="lora", T=2048, requests=5, K=4096, N=2048, R=64, L=8, dtype="bf16"),
        # a long chunk of several requests, of odd lengths, beside a product in float32
        dict(name="lora_long", op="lora", T=8191, requests=13, K=2048, N=4096, R=32, L=16, dtype="f32"),
        # the drafter's linear on one block of 16 positions
        dict(name="linear_block", op="linear", T=16, requests=1, K=2048, N=4096, R=16, L=8),
        # eight sequences' blocks, each with its own adapter
        dict(name="linear_blocks", op="linear", T=128, requests=8, K=2048, N=4096, R=16, L=8),
        # 64 sequences' blocks
        dict(name="linear_many", op="linear", T=1024, requests=64, K=2048, N=4096, R=32, L=48),
    ]


def _log_uniform(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("route", "route", "lora", "lora", "linear"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        size = rng.randint(2, 256 // groups)
        keep = rng.randint(1, groups)
        bias = rng.random() < 0.6
        return dict(op=op, T=_log_uniform(rng, 1, 16384), E=groups * size, topk=rng.randint(1, min(8, keep * size)),
                    score=rng.choice(("softmax", "sigmoid")), bias=bias, groups=groups, keep=keep,
                    top=rng.randint(1, 2), renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                    dtype=rng.choice(("f32", "bf16")), masked=rng.random() < 0.3)
    R = 8 * rng.choice((1, 2, 2, 3, 4, 8))
    L = _log_uniform(rng, 1, 64)
    if op == "lora":
        T = _log_uniform(rng, 1, 8191)
        return dict(op=op, T=T, requests=T if T <= 64 and rng.random() < 0.5 else _log_uniform(rng, 1, min(T, 64)),
                    K=8 * rng.randint(8, 256), N=_log_uniform(rng, 16, 4096), R=R, L=L,
                    dtype=rng.choice(("f32", "bf16")))
    requests = _log_uniform(rng, 1, 64)
    return dict(op=op, T=max(1, 16 * requests - rng.randint(0, 15)), requests=requests, K=128 * rng.randint(1, 16),
                N=16 * rng.randint(1, 256), R=R, L=L)


def _size(name):
    return 4 if name == "f32" else 2


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "route":
        E, k = c["E"], c["topk"]
        return {"bytes": T * E * _size(c["dtype"]) + (4 * E if c["bias"] else 0) + 16 * T * k + 4 * (E + 1),
                "flops": 2 * T * E}
    K, N, R, L = c["K"], c["N"], c["R"], c["L"]
    # seven requests in eight have an adapter; the adapters in use, on average
    used = L * (1.0 - (1.0 - 0.875 / L) ** c["requests"])
    adapters = used * R * (K + N) * 2 + 4 * T
    flops = 0.875 * 2 * T * R * (K + N)
    if c["op"] == "lora":
        return {"bytes": T * K * 2 + 2 * T * N * _size(c["dtype"]) + adapters, "flops": flops}
    return {"bytes": N * K + N * (K // 128) * 2 + T * K * 2 + T * N * 4 + adapters, "flops": 2 * T * K * N + flops}


# --------------------------------------------------------------------------------------------------------- the inputs

def _activations(g, rows, K):
    """N(0, 1) with one channel in a hundred twenty times larger, the same ones in every row, as bfloat16."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    n = round(0.01 * K)
    if n:
        x[:, torch.randperm(K, generator=g, device="cuda")[:n]] *= 20.0
    return x.to(torch.bfloat16)


def _adapters(g, c):
    """Adapters [L, R, K] and [L, N, R], their scales, and the adapter of each row: a request's rows lie together, one
    request in eight has no adapter (-1)."""
    T, n, L = c["T"], c["requests"], c["L"]
    a = (torch.randn((L, c["R"], c["K"]), generator=g, device="cuda") / math.sqrt(c["K"])).to(torch.bfloat16)
    b = (0.02 * torch.randn((L, c["N"], c["R"]), generator=g, device="cuda")).to(torch.bfloat16)
    scale = torch.exp2(torch.randint(0, 3, (L,), generator=g, device="cuda").float()) / 2
    which = torch.randint(0, L, (n,), generator=g, device="cuda")
    if n > 1:
        which = torch.where(torch.rand((n,), generator=g, device="cuda") < 0.125, torch.full_like(which, -1), which)
    if c["op"] == "linear":
        request = torch.arange(T, device="cuda") * n // T            # blocks of the same length
    else:
        cuts = torch.randperm(T - 1, generator=g, device="cuda")[:n - 1] + 1
        request = torch.zeros((T,), dtype=torch.int64, device="cuda")
        request[cuts] = 1
        request = request.cumsum(0)                                  # lengths by chance, one row at least
    return {"a": a, "b": b, "scale": scale, "adapter": which[request].to(torch.int32)}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        # skewed logits: some experts are liked by most tokens
        logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
        if c["masked"]:
            off = torch.rand((E,), generator=g, device="cuda") < 0.05
            pad = torch.rand((T,), generator=g, device="cuda") < 0.02
            logits = torch.where(off | pad.unsqueeze(-1), torch.full_like(logits, -math.inf), logits)
        s["logits"] = logits.to(_dtype(c["dtype"]))
        s["bias"] = 0.1 * torch.randn((E,), generator=g, device="cuda") if c["bias"] else None
        return s
    s["x"] = _activations(g, c["T"], c["K"])
    s.update(_adapters(g, c))
    if c["op"] == "lora":
        s["base"] = torch.randn((c["T"], c["N"]), generator=g, device="cuda").to(_dtype(c["dtype"]))
    else:
        s["codes"] = torch.randint(-127, 128, (c["N"], c["K"]), generator=g, device="cuda").to(torch.int8)
        s["scales"] = (torch.rand((c["N"], c["K"] // 128), generator=g, device="cuda") * 4e-4 + 1e-4).to(torch.float16)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _plain_route(s):
    c, l = s["case"], s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["topk"], c["groups"]
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(-1, keepdim=True)
        e = torch.where(l > -math.inf, torch.exp(l - top), torch.zeros_like(l))
        score = e / torch.where(top > -math.inf, e.sum(-1, keepdim=True), torch.ones_like(top))
    # without a bias the larger logit is the larger score
    choice = l if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        worth = choice if c["top"] == 1 or s["bias"] is not None else score
        worth = torch.sort(worth.view(T, G, E // G), dim=-1, descending=True).values[..., :c["top"]].sum(-1)
        best = torch.sort(worth, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        stays = (torch.arange(G, device=l.device).view(1, G, 1) == best.unsqueeze(1)).any(-1)
        stays = stays.unsqueeze(-1).expand(T, G, E // G).reshape(T, E)
        # experts of the other groups come after every one that stays, even after -inf
        order = torch.sort(choice, dim=-1, descending=True, stable=True).indices
        first = torch.sort(stays.gather(1, order).to(torch.int8), dim=-1, descending=True, stable=True).indices
        ids = order.gather(1, first[:, :k])
    else:
        ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    off = (flat.unsqueeze(0) < torch.arange(E + 1, device=flat.device).unsqueeze(1)).sum(-1)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return {"topk_ids": i32(ids), "topk_w": (w * c["scale"]).float(), "expert_off": i32(off),
            "sorted_pairs": i32(order), "pair_pos": i32(pos)}


def _plain_delta(s):
    """The adapters' part: every adapter's rank-R values, each row's own ones kept."""
    L, R, K = s["a"].shape
    h = s["x"].float() @ s["a"].float().view(L * R, K).t()
    mine = s["adapter"].long().unsqueeze(-1) == torch.arange(L, device=h.device)
    weight = torch.where(mine, s["scale"], torch.zeros_like(s["scale"]))
    h = (h.view(-1, L, R) * weight.unsqueeze(-1)).view(-1, L * R)
    return h @ s["b"].float().permute(0, 2, 1).reshape(L * R, -1)


def run(state):
    s, c = state, state["case"]
    if own:
        import int8_hadamard_domain_amd as i8h
        if c["op"] == "route":
            r = i8h.moe_route_scored_permute(s["logits"], c["topk"], score=c["score"], bias=s["bias"],
                                             groups=c["groups"], topk_groups=c["keep"], group_top=c["top"],
                                             renormalize=c["renorm"], scale=c["scale"])
            return {key: r[key] for key in ("topk_ids", "topk_w", "expert_off", "sorted_pairs", "pair_pos")}
        if c["op"] == "lora":
            return i8h.lora_add(s["base"], s["x"], s["a"], s["b"], s["adapter"], s["scale"])
        return i8h.linear_i8f16_lora(s["x"], s["codes"], s["scales"], s["a"], s["b"], s["adapter"], s["scale"])

    if c["op"] == "route":
        return _plain_route(s)
    if c["op"] == "lora":
        return (s["base"].float() + _plain_delta(s)).to(s["base"].dtype)
    w = (s["codes"].float().view(c["N"], -1, 128) * s["scales"].float().unsqueeze(-1)).view(c["N"], c["K"])
    return s["x"].float() @ w.t() + _plain_delta(s)


# ---------------------------------------------------------------------------- the definitions, once more, in 64 bits

def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "route":
        # the weights of the experts that the order of the definition picks, a row's own arithmetic in numpy
        import numpy as np
        l = s["logits"].double().cpu().numpy()
        T, E = l.shape
        if c["score"] == "sigmoid":
            e = np.exp(-np.abs(l))
            p = np.where(l >= 0, 1.0, e) / (1.0 + e)
        else:
            top = np.where(np.isfinite(l.max(1, keepdims=True)), l.max(1, keepdims=True), 0.0)
            e = np.exp(l - top)
            p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
        key = l if s["bias"] is None else p + s["bias"].double().cpu().numpy()
        if c["groups"] > 1:
            size = E // c["groups"]
            value = p if s["bias"] is None and c["top"] == 2 else key
            g = np.sort(value.reshape(T, -1, size), -1)[..., size - c["top"]:].sum(-1)
            lost = np.argsort(-g, 1, kind="stable")[:, c["keep"]:]
            out = np.zeros((T, c["groups"]), dtype=bool)
            np.put_along_axis(out, lost, True, 1)
            ids = np.lexsort((-key, out.repeat(size, 1)))[:, :c["topk"]]
        else:
            ids = np.argsort(-key, 1, kind="stable")[:, :c["topk"]]
        w = np.take_along_axis(p, ids, 1)
        if c["renorm"]:
            w = w / np.where(w.sum(1, keepdims=True) > 0, w.sum(1, keepdims=True), 1.0)
        return {"topk_ids": None, "topk_w": torch.from_numpy(w * c["scale"]).cuda(), "expert_off": None,
                "sorted_pairs": None, "pair_pos": None}
    x = s["x"].double()
    if c["op"] == "lora":
        y = s["base"].double()
    else:
        y = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device="cuda")
        for g in range(c["K"] // 128):
            cols = slice(128 * g, 128 * g + 128)
            y += (x[:, cols] @ s["codes"][:, cols].double().t()) * s["scales"][:, g].double()
    for l in s["adapter"].unique().tolist():
        if l >= 0:
            rows = (s["adapter"] == l).nonzero().squeeze(-1)
            h = x[rows] @ s["a"][l].double().t()
            y[rows] += s["scale"][l].double() * (h @ s["b"][l].double().t())
    return y

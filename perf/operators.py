"""The MXFP4 expert operators and the verification of drafted tokens: cases, inputs, plain forms.

Four operators, each through the package's public call (`own` true) or in plain torch (`own` false):

  quantise    mxfp4_quantize, then mxfp4_dequantize: values -> E2M1 codes with one E8M0 scale per 32 -> values
  gate_up     moe_gateup_mxfp4_grouped: grouped product of quantised activations with MXFP4 weights, GELU(gate) * up
  down        moe_down_mxfp4_combine: grouped product with the MXFP4 down projections, weighted merge per token
  verify      draft_verify: which drafted tokens stay, and the token sampled after them

MXFP4 (the OCP microscaling formats): a block of 32 values shares the scale 2^(s - 127) (byte s; 255 is NaN), each
value is a 4-bit E2M1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), two to a byte, the lower nibble first.
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # activations of one drafter block (16 positions) checked against their 4-bit form
        dict(name="quantise_block", op="quantise", rows=16, K=2048, dtype="bf16"),
        # one matrix of experts' weights packed on the device: 16 experts x 1536 rows
        dict(name="quantise_weights", op="quantise", rows=24576, K=2048, dtype="f32"),
        # one decoded token: latency
        dict(name="gate_up_decode", op="gate_up", T=1, K=2048, E=128, topk=8, N=1536, act="f32", pre=False),
        # a few sequences decoded together, an odd number, with the sums before the activation
        dict(name="gate_up_few", op="gate_up", T=7, K=1920, E=60, topk=4, N=1408, act="f32", pre=True),
        # a verify batch: 8 sequences x (1 + 15 drafted), few pairs an expert
        dict(name="gate_up_verify", op="gate_up", T=128, K=2048, E=128, topk=8, N=1536, act="bf16", pre=False),
        # a prefill chunk
        dict(name="gate_up_prefill", op="gate_up", T=2048, K=2048, E=128, topk=8, N=1536, act="bf16", pre=False),
        # the down projections behind them: one token, a verify batch on float32 rows, an odd prefill chunk
        dict(name="down_decode", op="down", T=1, I=768, E=128, topk=8, H=2048, act="f32"),
        dict(name="down_verify", op="down", T=128, I=768, E=128, topk=8, H=2048, act="f32"),
        dict(name="down_prefill", op="down", T=1999, I=768, E=128, topk=8, H=2048, act="bf16"),
        # one sequence, 15 drafted tokens, a large vocabulary: latency
        dict(name="verify_one", op="verify", B=1, D=15, V=262144, draft="probs"),
        # the verify batch's 8 sequences with an odd vocabulary, tokens drafted greedily (no draft distribution)
        dict(name="verify_greedy", op="verify", B=8, D=15, V=50257, draft="tokens"),
        # many sequences served together
        dict(name="verify_many", op="verify", B=64, D=7, V=131072, draft="probs"),
    ]


def _log_uniform(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("quantise", "gate_up", "gate_up", "down", "down", "verify"))
    if op == "quantise":
        return dict(op=op, rows=_log_uniform(rng, 1, 24576), K=_log_uniform(rng, 32, 2048, 32),
                    dtype=rng.choice(("bf16", "f32")))
    if op == "verify":
        B = _log_uniform(rng, 1, 64)
        return dict(op=op, B=B, D=rng.randint(0, 15 if B <= 16 else 7), V=_log_uniform(rng, 7, 131072),
                    draft=rng.choice(("probs", "tokens")))
    E = _log_uniform(rng, 1, 128)
    topk = rng.randint(1, min(E, 8))
    T = _log_uniform(rng, 1, 2048)
    if op == "gate_up":
        return dict(op=op, T=T, K=128 * rng.randint(1, 16), E=E, topk=topk, N=64 * rng.randint(1, 24),
                    act=rng.choice(("f32", "bf16")), pre=rng.random() < 0.25)
    return dict(op=op, T=T, I=32 * rng.randint(1, 24), E=E, topk=topk, H=32 * rng.randint(1, 64),
                act=rng.choice(("f32", "bf16")))


def _touched(c):
    """Experts that get at least one pair, on average."""
    return c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["op"] == "quantise":
        n = c["rows"] * c["K"]
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * size, "flops": 0}
    if c["op"] == "verify":
        # one row of each distribution a sequence (the row where it stops), and the short lists
        rows = 2 if c["draft"] == "probs" else 1
        return {"bytes": c["B"] * (rows * c["V"] * 4 + c["D"] * 24 + 16), "flops": 2 * c["B"] * c["V"]}
    P = c["T"] * c["topk"]
    size = 4 if c["act"] == "f32" else 2
    if c["op"] == "gate_up":
        N, K = c["N"], c["K"]
        weights = _touched(c) * N * (K / 2 + K / 32)
        out = P * (N // 2) * size + (P * N * 4 if c["pre"] else 0)
        return {"bytes": weights + c["T"] * K * 2 + out + P * 4 + (c["E"] + 1) * 4, "flops": 2 * P * N * K}
    H, I = c["H"], c["I"]
    weights = _touched(c) * H * (I / 2 + I / 32)
    return {"bytes": weights + P * I * size + c["T"] * H * 4 + P * 16 + (c["E"] + 1) * 4, "flops": 2 * P * H * I}


# --------------------------------------------------------------------------------------------------------- the inputs

def _pack(values, scale_bytes):
    """Multiples of the E2M1 grid [..., K] -> codes [..., K/2] uint8."""
    a = values.abs()
    code = (2 * a).clamp(max=4) + (a >= 3).float() + (a >= 4).float() + (a >= 6).float()
    code = code.to(torch.uint8) | (torch.signbit(values).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _weights(g, E, R, K):
    """MXFP4 weights [E, R, K] of N(0, 0.02^2) rows whose blocks differ in magnitude."""
    codes = torch.empty((E, R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, R, K // 32), dtype=torch.uint8, device="cuda")
    for e in range(0, E, 16):
        n = min(16, E - e)
        w = torch.randn((n, R, K), generator=g, device="cuda") * 0.02
        w = w * torch.exp2(torch.randint(-1, 2, (n, R, K // 32, 1), generator=g, device="cuda").float()).expand(
            n, R, K // 32, 32).reshape(n, R, K)
        q, s = _quantise(w)
        codes[e:e + n] = _pack(q, s)
        scales[e:e + n] = (s + 127).to(torch.uint8)
    return codes, scales


def _routing(g, T, E, topk):
    """The lists that moe_route_permute writes, of skewed router logits."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    w, ids = torch.topk(logits, topk, dim=-1)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    count = torch.bincount(flat, minlength=E)
    off = torch.cat([count.new_zeros(1), count.cumsum(0)])
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return {"topk_ids": i32(ids), "topk_w": torch.softmax(w, -1).float().contiguous(), "expert_off": i32(off),
            "sorted_pairs": i32(order), "pair_pos": i32(pos)}, int(count.max())


def _activations(g, rows, K, dtype):
    """N(0, 1) with one channel in a hundred twenty times larger, the same ones in every row."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    n = round(0.01 * K)
    if n:
        x[:, torch.randperm(K, generator=g, device="cuda")[:n]] *= 20.0
    return x.to(dtype)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quantise":
        s["x"] = _activations(g, c["rows"], c["K"], _dtype(c["dtype"]))
    elif c["op"] == "gate_up":
        s["x"] = _activations(g, c["T"], c["K"], torch.bfloat16)
        s["codes"], s["scales"] = _weights(g, c["E"], c["N"], c["K"])
        s["routing"], s["most"] = _routing(g, c["T"], c["E"], c["topk"])
    elif c["op"] == "down":
        # rows as GELU(gate) * up leaves them: small values with a heavy tail
        P = c["T"] * c["topk"]
        a = torch.randn((P, c["I"]), generator=g, device="cuda")
        s["act"] = (a * torch.randn((P, c["I"]), generator=g, device="cuda")).to(_dtype(c["act"]))
        s["codes"], s["scales"] = _weights(g, c["E"], c["H"], c["I"])
        s["routing"], s["most"] = _routing(g, c["T"], c["E"], c["topk"])
    else:
        B, D, V = c["B"], c["D"], c["V"]
        t = 3.0 * torch.randn((B, D + 1, V), generator=g, device="cuda")
        d = t[:, :D] + 0.7 * torch.randn((B, D, V), generator=g, device="cuda")
        s["p"] = torch.softmax(t, -1)
        if c["draft"] == "probs":
            s["q"] = torch.softmax(d, -1)
            d -= torch.log(-torch.log(torch.rand((B, D, V), generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
        else:
            s["q"] = None
        s["drafted"] = d.argmax(-1).to(torch.int32) if D else torch.empty((B, 0), dtype=torch.int32, device="cuda")
        s["u"] = torch.rand((B, D), generator=g, device="cuda")
        s["u_next"] = torch.rand((B,), generator=g, device="cuda")
        # most sequences use the whole draft, some a shorter one
        s["length"] = torch.minimum(torch.randint(0, 2 * D + 1, (B,), generator=g, device="cuda"),
                                    torch.full((B,), D, device="cuda")).to(torch.int32)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _quantise(x):
    """x [..., K] float32 -> (multiples of the E2M1 grid [..., K], exponents [..., K/32]); NaN where a block has one."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.clamp(torch.frexp(top).exponent - 3, min=-127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    y = torch.ldexp(b, -e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(torch.clamp(torch.round(a / step) * step, max=6.0), y)
    q = torch.where(torch.isfinite(top), q, torch.full_like(q, math.nan))
    return q.reshape(x.shape), e.squeeze(-1)


def _times_scale(q, e):
    return torch.ldexp(q.reshape(*e.shape, 32), e.unsqueeze(-1)).reshape(q.shape)


def _unpack(codes, scales):
    """Codes [..., K/2] and scale bytes [..., K/32] -> float32 values [..., K]."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    pairs = torch.stack([v.repeat(16), v.repeat_interleave(16)], -1)
    q = torch.index_select(pairs, 0, codes.reshape(-1).to(torch.int32))
    q = q.reshape(*codes.shape[:-1], -1)
    return _times_scale(q, scales.to(torch.int32) - 127)


def _grouped(rows, codes, scales, routing, most):
    """rows [P, K] in expert order times their expert's weights [R, K]: [P, R] float32."""
    off = routing["expert_off"].long()
    P, E = rows.shape[0], codes.shape[0]
    r = torch.arange(P, device=rows.device)
    e = torch.searchsorted(off[1:], r, right=True)
    if P <= E:   # few rows: each row's own weights
        return torch.bmm(_unpack(codes[e], scales[e]), rows.unsqueeze(-1)).squeeze(-1)
    padded = rows.new_zeros((E, most, rows.shape[1]))
    padded[e, r - off[e]] = rows
    y = torch.bmm(padded, _unpack(codes, scales).transpose(1, 2).contiguous())
    return y[e, r - off[e]]


def _gelu_tanh(x):
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _plain_verify(s):
    p, q, drafted, u = s["p"], s["q"], s["drafted"].long(), s["u"].double()
    B, D1, V = p.shape
    D = D1 - 1
    length = s["length"].long()
    at = torch.arange(B, device=p.device)
    pt = p[:, :D].gather(2, drafted.unsqueeze(-1)).squeeze(-1).double()
    qt = torch.ones_like(pt) if q is None else q.gather(2, drafted.unsqueeze(-1)).squeeze(-1).double()
    keep = (u * qt < pt) & (torch.arange(D, device=p.device) < length.unsqueeze(-1))
    n = torch.cumprod(keep.long(), -1).sum(-1)
    row = p[at, n].double()
    rest = row
    if D:
        stopped = (n < length).unsqueeze(-1)
        m = n.clamp(max=D - 1)
        if q is None:
            other = torch.arange(V, device=p.device) == drafted[at, m].unsqueeze(-1)
            less = torch.where(other, 0.0, row)
        else:
            less = torch.clamp(row - q[at, m].double(), min=0.0)
        rest = torch.where(stopped, less, row)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, row)
    upto = rest.cumsum(-1)
    nxt = (upto <= s["u_next"].double().unsqueeze(-1) * upto[:, -1:]).sum(-1).clamp(max=V - 1)
    i = torch.arange(D + 1, device=p.device)
    tokens = torch.full((B, D + 1), -1, dtype=torch.int64, device=p.device)
    tokens[:, :D] = drafted
    tokens = torch.where(i < n.unsqueeze(-1), tokens, torch.full_like(tokens, -1))
    tokens[at, n] = nxt
    return {"tokens": tokens.to(torch.int32), "accepted": n.to(torch.int32)}


def run(state):
    s, c = state, state["case"]
    if own:
        import int8_hadamard_domain_amd as i8h
        if c["op"] == "quantise":
            return i8h.mxfp4_dequantize(*i8h.mxfp4_quantize(s["x"]), dtype=s["x"].dtype)
        if c["op"] == "gate_up":
            r = s["routing"]
            pre, act = i8h.moe_gateup_mxfp4_grouped(s["x"], s["codes"], s["scales"], c["topk"], r["expert_off"],
                                                    r["sorted_pairs"], gate_up=c["pre"], act_dtype=_dtype(c["act"]))
            return {"act": act, "pre": pre} if c["pre"] else {"act": act}
        if c["op"] == "down":
            return i8h.moe_down_mxfp4_combine(s["act"], s["codes"], s["scales"], s["routing"])
        tokens, accepted = i8h.draft_verify(s["p"], s["q"], s["drafted"], s["u"], s["u_next"], draft_len=s["length"])
        return {"tokens": tokens, "accepted": accepted}

    if c["op"] == "quantise":
        return _times_scale(*_quantise(s["x"].float())).to(s["x"].dtype)
    if c["op"] == "gate_up":
        r = s["routing"]
        x = _times_scale(*_quantise(s["x"].float()))
        pre = _grouped(x[r["sorted_pairs"].long() // c["topk"]], s["codes"], s["scales"], r, s["most"])
        gate, up = pre.chunk(2, -1)
        act = (_gelu_tanh(gate) * up).to(_dtype(c["act"]))
        return {"act": act, "pre": pre} if c["pre"] else {"act": act}
    if c["op"] == "down":
        r = s["routing"]
        a = _times_scale(*_quantise(s["act"].float()))
        y = _grouped(a, s["codes"], s["scales"], r, s["most"])
        return (r["topk_w"].unsqueeze(-1) * y[r["pair_pos"].long()].view(c["T"], c["topk"], -1)).sum(1)
    return _plain_verify(s)


# ---------------------------------------------------------------------------- the definitions, once more, in 64 bits

def _exact_value(codes, scales):
    """MXFP4 values from the fields of each code: sign, two exponent bits, one mantissa bit."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).long()
    sign, ex, man = 1.0 - 2.0 * (c >> 3).double(), ((c >> 1) & 3).double(), (c & 1).double()
    v = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2(ex - 1))
    return sign * v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_quantise(x):
    """The value that each x is held as: the nearest grid point, the even code in a tie."""
    x = x.double().reshape(*x.shape[:-1], -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.clamp(torch.floor(torch.log2(top)) - 2, min=-127.0))
    # log2 may sit on the wrong side of a power of two: the largest value lies in [4, 8) scales
    scale = torch.where(top >= 8 * scale, 2 * scale, scale)
    scale = torch.where((top < 4 * scale) & (scale > 2.0 ** -127), scale / 2, scale)
    y = x.abs() / scale
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    # a value on a border goes to the even code: up from the odd borders' lower side only
    code = (y.unsqueeze(-1) > borders).sum(-1) + ((y.unsqueeze(-1) == borders[1::2]).any(-1)).long()
    v = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[code]
    return (torch.copysign(v, x) * scale).reshape(*x.shape[:-2], -1)


def exact(case, seed):
    c = dict(case)
    if c["op"] == "verify":
        return None   # whole numbers
    s = prepare(case, seed)
    if c["op"] == "quantise":
        return torch.cat([_exact_quantise(v) for v in s["x"].split(2048)])
    off = s["routing"]["expert_off"].tolist()
    if c["op"] == "gate_up":
        x = _exact_quantise(s["x"])[s["routing"]["sorted_pairs"].long() // c["topk"]]
    else:
        x = torch.cat([_exact_quantise(v) for v in s["act"].split(2048)])
    y = torch.zeros((x.shape[0], s["codes"].shape[1]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        if off[e + 1] > off[e]:
            y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ _exact_value(s["codes"][e], s["scales"][e]).t().contiguous()
    if c["op"] == "gate_up":
        half = c["N"] // 2
        gate = y[:, :half]
        z = math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate ** 3)
        act = gate / (1.0 + torch.exp(-2.0 * z)) * y[:, half:]
        return {"act": act, "pre": y} if c["pre"] else {"act": act}
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    w = s["routing"]["topk_w"].double()
    pos = s["routing"]["pair_pos"].long().view(c["T"], c["topk"])
    for j in range(c["topk"]):
        out += w[:, j:j + 1] * y[pos[:, j]]
    return out

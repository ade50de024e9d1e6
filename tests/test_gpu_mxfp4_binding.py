"""The binding of the MXFP4 and draft-verification calls rejects tensors that
do not fit with TypeError or ValueError before anything is launched. Each case
changes one tensor of an otherwise valid call."""

import pytest
import torch

import int8_hadamard_domain_amd as i8h

pytestmark = pytest.mark.gpu

T, K, E, N, H, k = 99, 256, 8, 128, 64, 2


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8, device="cuda")


@pytest.fixture(scope="module")
def inp(gpu_available):
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    r = i8h.moe_route_permute(torch.randn((T, E), device="cuda"), k)
    return x, r


def _raises(fn, *a, **kw):
    with pytest.raises((TypeError, ValueError)):
        fn(*a, **kw)


def test_quantiser(inp):
    x = inp[0]
    _raises(i8h.mxfp4_quantize, x[:, :48].contiguous())
    _raises(i8h.mxfp4_quantize, x[:, ::2])
    _raises(i8h.mxfp4_quantize, x.half())
    _raises(i8h.mxfp4_quantize, torch.tensor(1.0, device="cuda"))
    _raises(i8h.mxfp4_quantize, x, codes=u8(T, K))
    _raises(i8h.mxfp4_quantize, x, scales=u8(T, K // 16))
    _raises(i8h.mxfp4_quantize, x, codes=u8(T, K // 2).cpu())
    _raises(i8h.mxfp4_dequantize, u8(T, 24), u8(T, 1))
    _raises(i8h.mxfp4_dequantize, u8(T, 32), u8(T, 1))
    _raises(i8h.mxfp4_dequantize, u8(T, 32), u8(T, 2), dtype=torch.float16)
    _raises(i8h.mxfp4_dequantize, u8(T, 32), u8(T, 2), out=torch.empty((T, 32), device="cuda"))


def test_gate_up(inp):
    x, r = inp
    off, sp = r["expert_off"], r["sorted_pairs"]
    f = i8h.moe_gateup_mxfp4_grouped
    c, s = u8(E, N, K // 2), u8(E, N, K // 32)
    _raises(f, x.float(), c, s, k, off, sp)
    _raises(f, x, u8(E, N, K), s, k, off, sp)
    _raises(f, x, c, u8(E, N, K // 16), k, off, sp)
    _raises(f, x, c.view(torch.int8), s, k, off, sp)
    _raises(f, x, c, s.cpu(), k, off, sp)
    _raises(f, x, c, s, k + 1, off, sp)
    _raises(f, x, c, s, k, off[:-1].contiguous(), sp)
    _raises(f, x, c, s, k, off, sp.long())
    _raises(f, x, c, s, k, off, sp, act_dtype=torch.float16)
    _raises(f, x, c, s, k, off, sp, act=torch.empty((T * k, N), device="cuda"))
    _raises(f, x, c, s, k, off, sp, gate_up=torch.empty((T * k, N), dtype=torch.bfloat16, device="cuda"))
    _raises(f, x, c, s, k, off, sp, workspace=u8(16))
    with pytest.raises(i8h.I8HError) as e:
        f(x, u8(E, 96, K // 2), u8(E, 96, K // 32), k, off, sp)
    assert e.value.status == i8h.I8H_EUNSUPPORTED
    with pytest.raises(i8h.I8HError) as e:                       # a view that starts off a 16-byte border
        buf = torch.zeros(T * K + 1, dtype=torch.bfloat16, device="cuda")
        f(buf[1:].view(T, K), c, s, k, off, sp)
    assert e.value.status == i8h.I8H_EINVAL


def test_down(inp):
    r = inp[1]
    f = i8h.moe_down_mxfp4_combine
    act, c, s = torch.randn((T * k, N // 2), device="cuda"), u8(E, H, N // 4), u8(E, H, N // 64)
    _raises(f, act.half(), c, s, r)
    _raises(f, act[:-1].contiguous(), c, s, r)
    _raises(f, act, u8(E, H, N // 2), s, r)
    _raises(f, act, c, u8(E, H, 1), r)
    _raises(f, act, c, s, r, out=torch.empty((T, H + 1), device="cuda"))
    _raises(f, act, c, s, r, workspace=u8(16))
    _raises(f, act, c, s, dict(r, pair_pos=r["pair_pos"][:-1].contiguous()))
    _raises(f, act, c, s, dict(r, expert_off=r["expert_off"][:-1].contiguous()))
    assert f(act, c, s, r).shape == (T, H)


def test_draft(inp):
    B, D, V = 2, 3, 40
    f = i8h.draft_verify
    p, q = torch.rand((B, D + 1, V), device="cuda"), torch.rand((B, D, V), device="cuda")
    x = torch.zeros((B, D), dtype=torch.int32, device="cuda")
    u, un = torch.rand((B, D), device="cuda"), torch.rand(B, device="cuda")
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    _raises(f, p.double(), q, x, u, un)
    _raises(f, p[:, :0].contiguous(), q, x, u, un)
    _raises(f, p[:, :, ::2], q, x, u, un)
    _raises(f, p, q.bfloat16(), x, u, un)
    _raises(f, p, q[:, :-1].contiguous(), x, u, un)
    _raises(f, p, q, x.long(), u, un)
    _raises(f, p, q, x, u[:, :-1].contiguous(), un)
    _raises(f, p, q, x, u, un.double())
    _raises(f, p, q, x, u, un, draft_len=n.long())
    _raises(f, p, q, x, u, un, tokens=torch.zeros((B, D), dtype=torch.int32, device="cuda"))
    _raises(f, p, q, x, u, un, accepted=n[:1].contiguous())
    _raises(f, p, q, x, u, un, workspace=u8(8))
    assert f(p, q, x, u, un, draft_len=n)[0].shape == (B, D + 1)

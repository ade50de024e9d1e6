"""Host-side checks of the scored routing and adapter entry points (no GPU):
every declared function is exported, invalid arguments are refused with the
documented status codes before anything is launched (dummy addresses that are
never read), and the binding refuses tensors that do not fit."""

import ctypes
import os
import re

import pytest
import torch

import int8_hadamard_domain_amd as i8h

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
EINVAL, EUNSUP, OK = i8h.I8H_EINVAL, i8h.I8H_EUNSUPPORTED, i8h.I8H_OK
P = ctypes.c_void_p
A = [P((i + 1) << 40) for i in range(16)]     # 256-byte aligned dummy addresses far apart, never touched
ODD, BYTE, EIGHT = P((99 << 40) + 2), P((99 << 40) + 1), P((99 << 40) + 8)
MAX = (1 << 31) - 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(i8h.LIB_PATH):
        pytest.skip("libi8h.so not built")
    return i8h.lib()


@pytest.mark.parametrize("header", ["i8h_scored.h", "i8h_lora.h"])
def test_every_declared_function_is_exported_and_bound(L, header):
    with open(os.path.join(INCLUDE, header)) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b([a-z][a-z0-9_]*)\s*\(", src)) - {"defined"}
    assert names
    for n in names:
        assert getattr(L, n).argtypes is not None, n
        if not n.endswith("_workspace_size"):
            assert callable(getattr(i8h, n))


def test_scored_routing_validation(L):
    need = L.moe_route_scored_workspace_size(999, 64, 4)
    assert need > 0 and need % 256 == 0
    assert L.moe_route_scored_workspace_size(0, 64, 4) == 0 and L.moe_route_scored_workspace_size(5, 1025, 4) == 0

    def call(l=A[0], t=0, T=999, E=64, k=4, score=1, bias=A[1], g=8, kg=4, top=2, ren=1, scale=1.0, ids=A[2], w=A[3],
             off=A[4], sp=A[5], pos=A[6], ws=A[7], wsb=need):
        return L.moe_route_scored_permute(l, t, T, E, k, score, bias, g, kg, top, ren, scale, ids, w, off, sp, pos, ws,
                                          wsb, None)
    for bad in (dict(t=2), dict(t=-1), dict(T=-1), dict(E=0), dict(k=0), dict(score=2), dict(score=-1), dict(g=0),
                dict(g=7), dict(g=-8), dict(kg=0), dict(kg=9), dict(top=0), dict(top=3), dict(g=64, kg=64),
                dict(kg=1, k=9), dict(k=65, kg=8), dict(l=None), dict(ids=None), dict(w=None), dict(off=None),
                dict(sp=None), dict(pos=None), dict(ws=None), dict(l=ODD), dict(l=BYTE, t=1), dict(bias=ODD),
                dict(ids=ODD), dict(w=ODD), dict(off=ODD), dict(sp=ODD), dict(pos=ODD), dict(ws=EIGHT),
                dict(wsb=need - 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(E=2048), dict(k=33, kg=8), dict(E=130, g=65, kg=65, k=2), dict(T=MAX), dict(T=1 << 29),
                dict(T=MAX, E=1024, k=1)):
        assert call(**bad) == EUNSUP, bad
    assert call(T=0) == OK and call(T=0, l=None, ws=None, wsb=0) == OK


def lora_kwargs(need):
    return dict(base=A[0], bt=0, ldb=100, x=A[1], ldx=64, T=300, K=64, N=100, a=A[2], b=A[3], L_=3, R=16, ad=A[4],
                sc=A[5], out=A[6], ldo=100, ws=A[7], wsb=need)


def test_lora_add_validation(L):
    need = L.lora_add_workspace_size(300, 16)
    assert need >= 300 * 16 * 4 and need % 256 == 0 and need == L.lora_workspace_size(300, 16)
    assert L.lora_workspace_size(0, 16) == 0 and L.lora_workspace_size(9, 0) == 0 and L.lora_add_workspace_size(0, 0) == 0
    # few rows take none
    assert L.lora_add_workspace_size(64, 64) == 0 and L.lora_add_workspace_size(64, 72) > 0
    assert L.lora_add_workspace_size(65, 64) > 0 and L.lora_add_workspace_size(256, 16) == 0
    assert L.lora_add_workspace_size(257, 8) > 0 and L.lora_workspace_size(9, 16) > 0

    def call(**kw):
        v = dict(lora_kwargs(need), **kw)
        return L.lora_add(v["base"], v["bt"], v["ldb"], v["x"], v["ldx"], v["T"], v["K"], v["N"], v["a"], v["b"],
                          v["L_"], v["R"], v["ad"], v["sc"], v["out"], v["ldo"], v["ws"], v["wsb"], None)
    for bad in (dict(bt=2), dict(bt=-1), dict(T=-1), dict(K=0), dict(K=60), dict(N=0), dict(L_=0), dict(R=0),
                dict(R=12), dict(R=-8), dict(ldb=99), dict(ldo=99), dict(ldx=56), dict(ldx=68), dict(base=None),
                dict(x=None), dict(a=None), dict(b=None), dict(ad=None), dict(sc=None), dict(out=None), dict(ws=None),
                dict(x=EIGHT), dict(a=EIGHT), dict(b=EIGHT), dict(ad=ODD), dict(sc=ODD), dict(base=ODD), dict(out=ODD),
                dict(base=BYTE, bt=1), dict(out=BYTE, bt=1), dict(ws=EIGHT), dict(wsb=need - 1)):
        assert call(**bad) == EINVAL, bad
    # out may be base, with the same rows; it may meet no other input, nor base in part
    for bad in (dict(out=A[0], ldo=104), dict(out=P(A[0].value + 4)), dict(out=P(A[0].value - 4)), dict(out=A[1]),
                dict(out=A[2]), dict(out=A[3]), dict(out=A[4]), dict(out=A[5]), dict(out=A[7]),
                dict(out=P(A[1].value - 4 * 29999)), dict(out=P(A[2].value + 2 * 3 * 16 * 64 - 4))):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(R=264), dict(N=(1 << 22) + 1, ldb=1 << 23, ldo=1 << 23), dict(T=(1 << 26) + 1), dict(T=MAX)):
        assert call(**bad) == EUNSUP, bad
    assert call(T=0) == OK and call(T=0, x=None, out=None, ws=None) == OK


def test_linear_lora_validation(L):
    need = L.lora_workspace_size(9, 16)

    def call(x=A[1], T=9, K=128, c=A[0], s=A[6], N=48, a=A[2], b=A[3], L_=3, R=16, ad=A[4], sc=A[5], y=A[8], ws=A[7],
             wsb=need):
        return L.linear_i8f16_lora(x, T, K, c, s, N, a, b, L_, R, ad, sc, y, ws, wsb, None)
    for bad in (dict(T=-1), dict(K=0), dict(K=64), dict(N=0), dict(N=40), dict(L_=0), dict(R=0), dict(R=4),
                dict(x=None), dict(c=None), dict(s=None), dict(a=None), dict(b=None), dict(ad=None), dict(sc=None),
                dict(y=None), dict(ws=None), dict(x=EIGHT), dict(c=EIGHT), dict(s=BYTE), dict(a=EIGHT), dict(b=EIGHT),
                dict(ad=ODD), dict(sc=ODD), dict(y=ODD), dict(ws=EIGHT), dict(wsb=need - 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(y=A[0]), dict(y=A[1]), dict(y=A[2]), dict(y=A[3]), dict(y=A[4]), dict(y=A[5]), dict(y=A[6]),
                dict(y=A[7])):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(R=264), dict(N=(1 << 22) + 16), dict(T=1 << 24), dict(T=1 << 21, N=1 << 15)):
        assert call(**bad) == EUNSUP, bad
    assert call(T=0) == OK


def test_binding_refuses_tensors_off_the_gpu():
    f32, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    with pytest.raises(ValueError, match="GPU"):
        i8h.moe_route_scored_permute(torch.zeros(3, 8), 2)
    with pytest.raises(TypeError):
        i8h.moe_route_scored_permute(torch.zeros(3, 8, dtype=torch.float16), 2)
    with pytest.raises(TypeError):
        i8h.moe_route_scored_permute([[0.0]], 1)
    args = [torch.zeros(2, 16), torch.zeros(2, 64, dtype=bf), torch.zeros(1, 8, 64, dtype=bf),
            torch.zeros(1, 16, 8, dtype=bf), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=f32)]
    with pytest.raises(ValueError, match="GPU"):
        i8h.lora_add(*args)
    with pytest.raises(TypeError):
        i8h.lora_add(torch.zeros(2, 16, dtype=torch.float64), *args[1:])
    with pytest.raises(ValueError, match="GPU"):
        i8h.linear_i8f16_lora(args[1], torch.zeros(16, 64, dtype=torch.int8), torch.zeros(16, 0), *args[2:])


def test_limits(L):
    """The documented limits: at them a call is taken (shown with T = 0), past them it is refused."""
    need = L.lora_workspace_size(300, 16)

    def add(**kw):
        v = dict(lora_kwargs(need), **kw)
        return L.lora_add(v["base"], v["bt"], v["ldb"], v["x"], v["ldx"], v["T"], v["K"], v["N"], v["a"], v["b"],
                          v["L_"], v["R"], v["ad"], v["sc"], v["out"], v["ldo"], v["ws"], v["wsb"], None)
    m = 1 << 22
    for ok, bad in ((dict(K=m, ldx=m), dict(K=m + 8, ldx=m + 8)), (dict(N=m, ldb=m, ldo=m), dict(N=m + 1, ldb=m + 1, ldo=m + 1)),
                    (dict(ldb=1 << 24), dict(ldb=(1 << 24) + 1)), (dict(ldo=1 << 24), dict(ldo=(1 << 24) + 1)),
                    (dict(ldx=1 << 24), dict(ldx=(1 << 24) + 8)), (dict(R=256), dict(R=264)),
                    (dict(), dict(T=(1 << 13) + 1, N=m, ldb=m, ldo=m))):
        assert add(T=0, **ok) == OK and add(**bad) == EUNSUP, (ok, bad)

    def linear(T, K, N, R):
        return L.linear_i8f16_lora(A[1], T, K, A[0], A[6], N, A[2], A[3], 3, R, A[4], A[5], A[8], A[7], need, None)
    assert linear(0, m, m, 256) == OK
    for bad in ((9, m + 128, 48, 16), (9, 128, m + 16, 16), (9, 128, 48, 264), (512, m, 48, 16), ((1 << 20) + 1, 128, 1 << 15, 16)):
        assert linear(*bad) == EUNSUP, bad
    for T, R in ((1, 8), (64, 64), (1 << 20, 256), ((1 << 26), 256)):
        assert L.lora_workspace_size(T, R) >= 4 * T * R


def _falls(sizes):
    return [(i, a, b) for i, (a, b) in enumerate(zip(sizes, sizes[1:])) if b < a]


def test_workspace_sizes_never_fall(L):
    """A workspace for the largest batch serves every smaller one, and one for the most experts, choices or the highest
    rank every lower: the sizes do not fall as any of these grow (lora_add's own are 0 or the common one)."""
    ts = sorted(set(range(1, 3000)) | {64 * i + d for i in range(40, 600) for d in (-1, 0, 1)} |
                {b + d for b in (1 << 14, 16640, 32768, 65536, 1 << 20, 1 << 24) for d in (-1, 0, 1, 2)})
    for R in (8, 32, 256):
        sizes = [L.lora_workspace_size(T, R) for T in ts]
        assert not _falls(sizes), (R, _falls(sizes)[:3])
        assert all(s >= 4 * T * R for s, T in zip(sizes, ts))
        own = [L.lora_add_workspace_size(T, R) for T in ts]
        assert not _falls(own) and all(o in (0, s) for o, s in zip(own, sizes))
    for T in (1, 64, 65, 256, 300, 5000):
        assert not _falls([L.lora_workspace_size(T, R) for R in range(8, 264, 8)])
        assert not _falls([L.lora_add_workspace_size(T, R) for R in range(8, 264, 8)])
    for E in (1, 16, 60, 256, 257, 384, 1024):
        for k in (1, 2, 5, 8, 9, 20, 32):
            sizes = [L.moe_route_scored_workspace_size(T, E, k) for T in ts]
            assert not _falls(sizes), (E, k, _falls(sizes)[:3])
    for T in (1, 33, 256, 257, 300, 1999, 4097, 16384, 16385, 70000):
        for k in (1, 8, 32):
            sizes = [L.moe_route_scored_workspace_size(T, E, k) for E in range(1, 1025)]
            assert not _falls(sizes), (T, k, _falls(sizes)[:3])
        for E in (16, 256, 1024):
            sizes = [L.moe_route_scored_workspace_size(T, E, k) for k in range(1, 33)]
            assert not _falls(sizes), (T, E, _falls(sizes)[:3])


def test_scored_routing_limits(L):
    """The documented limits, from both sides (a call within them gets as far as the missing logits)."""
    def call(T, E, k, groups=1, keep=1, top=1):
        return L.moe_route_scored_permute(None, 0, T, E, k, 0, None, groups, keep, top, 1, 1.0, A[2], A[3], A[4], A[5], A[6],
                                          A[7], 1 << 62, None)
    for k in (1, 3, 8, 9, 20, 32):
        most = ((1 << 22) - 1) * min(64, 512 // k)
        assert call(most, 1024, k) == EINVAL and call(most + 1, 1024, k) == EUNSUP, k
    assert call(5, 1024, 32, 64, 64) == EINVAL and call(5, 1025, 4) == EUNSUP and call(5, 1024, 33) == EUNSUP
    # one group: its worth decides nothing, and group_top is not held against its size
    assert call(0, 1, 1, top=2) == OK and call(0, 2, 1, 2, 1, top=2) == EINVAL

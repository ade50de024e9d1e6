"""Host-side checks of the MXFP4 and draft-verification entry points (no GPU):
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
A = ctypes.c_void_p(0x10000)      # a 256-byte aligned dummy address, never touched
ODD = ctypes.c_void_p(0x10002)    # misaligned for 4- and 16-byte data
BYTE = ctypes.c_void_p(0x10001)   # misaligned for everything but bytes
EIGHT = ctypes.c_void_p(0x10008)  # misaligned for 16-byte data
BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(i8h.LIB_PATH):
        pytest.skip("libi8h.so not built")
    return i8h.lib()


@pytest.mark.parametrize("header", ["i8h_mxfp4.h", "i8h_draft.h"])
def test_every_declared_function_is_exported_and_bound(L, header):
    with open(os.path.join(INCLUDE, header)) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b([a-z][a-z0-9_]*)\s*\(", src)) - {"defined"}
    assert names
    for n in names:
        assert getattr(L, n).argtypes is not None, n
        if not n.endswith("_workspace_size"):
            assert callable(getattr(i8h, n))


@pytest.mark.parametrize("name", ["mxfp4_quantize", "mxfp4_dequantize"])
def test_quantiser_validation(L, name):
    def call(x=A, t=0, T=4, K=64, c=A, s=A):
        if name == "mxfp4_quantize":
            return L.mxfp4_quantize(x, t, T, K, c, s, None)
        return L.mxfp4_dequantize(c, s, T, K, x, t, None)
    assert call(t=2) == EINVAL and call(t=-1) == EINVAL
    assert call(T=-1) == EINVAL and call(K=0) == EINVAL and call(K=48) == EINVAL and call(K=-32) == EINVAL
    assert call(x=None) == EINVAL and call(c=None) == EINVAL and call(s=None) == EINVAL
    assert call(x=EIGHT) == EINVAL and call(c=EIGHT) == EINVAL
    assert call(T=(1 << 31) - 1, K=2048) == EUNSUP          # more threads than a launch takes
    assert call(T=1 << 24, K=2048) == EUNSUP and call(T=1 << 30, K=32) == EUNSUP
    assert call(T=0) == OK and call(T=0, x=None, c=None, s=None) == OK


def test_gateup_validation(L):
    assert L.moe_gateup_mxfp4_workspace_size(8, 256, 4, 2) == 0        # one launch, no workspace
    assert L.moe_gateup_mxfp4_workspace_size(16, 256, 4, 2) == 0
    need = L.moe_gateup_mxfp4_workspace_size(99, 256, 4, 2)
    assert need > 99 * 256 * 17 // 32 and need % 256 == 0      # the quantised rows and a list
    assert L.moe_gateup_mxfp4_workspace_size(0, 256, 4, 2) == 0
    assert L.moe_gateup_mxfp4_workspace_size(99, 100, 4, 2) == 0

    def call(x=A, T=99, K=256, c=A, s=A, E=4, N=128, k=2, off=A, sp=A, gu=A, act=A, t=0, ws=A, wsb=need):
        return L.moe_gateup_mxfp4_grouped(x, T, K, c, s, E, N, k, off, sp, gu, act, t, ws, wsb, None)
    for bad in (dict(T=-1), dict(K=0), dict(K=96), dict(E=0), dict(N=0), dict(N=127), dict(k=0), dict(t=2),
                dict(x=None), dict(c=None), dict(s=None), dict(off=None), dict(sp=None), dict(x=EIGHT), dict(c=EIGHT),
                dict(s=ODD), dict(off=ODD), dict(sp=ODD), dict(gu=EIGHT), dict(act=EIGHT), dict(ws=None),
                dict(ws=EIGHT), dict(wsb=need - 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(N=96), dict(E=1025), dict(k=5), dict(E=64, k=33), dict(T=1 << 28, k=32, E=64), dict(T=1 << 25)):
        assert call(**bad) == EUNSUP, bad
    assert call(T=0) == OK and call(gu=None, act=None) == OK


def test_down_validation(L):
    assert L.moe_down_mxfp4_workspace_size(8, 96, 4, 64, 2) == 0
    small = L.moe_down_mxfp4_workspace_size(9, 96, 4, 64, 2)
    assert small >= 18 * 64 * 4 and small % 256 == 0          # y
    need = L.moe_down_mxfp4_workspace_size(99, 96, 4, 64, 2)
    assert need > 198 * 96 * 17 // 32 + 198 * 64 * 4 and need % 256 == 0      # quantised rows, y and a list
    assert L.moe_down_mxfp4_workspace_size(0, 96, 4, 64, 2) == 0
    assert L.moe_down_mxfp4_workspace_size(99, 100, 4, 64, 2) == 0

    def call(a=A, t=0, T=99, I=96, c=A, s=A, E=4, H=64, k=2, ids=A, w=A, off=A, pos=A, out=A, ws=A, wsb=need):
        return L.moe_down_mxfp4_combine(a, t, T, I, c, s, E, H, k, ids, w, off, pos, out, ws, wsb, None)
    for bad in (dict(T=-1), dict(I=0), dict(I=48), dict(E=0), dict(H=0), dict(H=36), dict(k=0), dict(t=2),
                dict(a=None), dict(c=None), dict(s=None), dict(ids=None), dict(w=None), dict(off=None), dict(pos=None),
                dict(out=None), dict(a=EIGHT), dict(c=EIGHT), dict(s=ODD), dict(ids=ODD), dict(w=ODD), dict(off=ODD),
                dict(pos=ODD), dict(out=EIGHT), dict(ws=None), dict(ws=EIGHT), dict(wsb=need - 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(H=72), dict(E=1025), dict(k=5), dict(E=64, k=33), dict(T=1 << 28, k=32, E=64), dict(T=1 << 25),
                dict(H=1 << 25, I=32), dict(H=1 << 25, I=96), dict(H=1 << 24, I=256)):
        assert call(**bad) == EUNSUP, bad
    assert call(T=0) == OK


def test_draft_validation(L):
    need = L.draft_verify_workspace_size(3, 5000)
    assert need > 0 and need % 256 == 0
    assert L.draft_verify_workspace_size(0, 5000) == 0 and L.draft_verify_workspace_size(3, 0) == 0

    def call(p=A, q=A, t=0, x=A, ln=A, u=A, un=A, B=3, D=4, V=5000, tok=A, acc=A, ws=A, wsb=need):
        return L.draft_verify(p, q, t, x, ln, u, un, B, D, V, tok, acc, ws, wsb, None)
    for bad in (dict(t=2), dict(B=-1), dict(D=-1), dict(V=0), dict(p=None), dict(x=None), dict(u=None), dict(un=None),
                dict(tok=None), dict(acc=None), dict(p=ODD), dict(q=ODD), dict(p=BYTE, t=1), dict(q=BYTE, t=1),
                dict(x=ODD), dict(ln=ODD), dict(u=ODD), dict(un=ODD), dict(tok=ODD), dict(acc=ODD), dict(ws=None),
                dict(ws=EIGHT), dict(wsb=need - 1)):
        assert call(**bad) == EINVAL, bad
    assert call(D=1024) == EUNSUP and call(B=65536, wsb=BIG) == EUNSUP
    assert call(B=0) == OK


def test_binding_refuses_what_does_not_fit():
    """On CPU tensors: the first check that fails says so; nothing reaches the library."""
    with pytest.raises(TypeError):
        i8h.mxfp4_quantize(torch.zeros((2, 32), dtype=torch.float16))
    with pytest.raises(TypeError):
        i8h.mxfp4_quantize([1.0] * 32)
    with pytest.raises(ValueError):
        i8h.mxfp4_quantize(torch.zeros((2, 32)))                       # not on the GPU
    with pytest.raises(ValueError):
        i8h.mxfp4_dequantize(torch.zeros((2, 16), dtype=torch.uint8), torch.zeros((2, 1), dtype=torch.uint8))
    with pytest.raises(ValueError):
        i8h.moe_gateup_mxfp4_grouped(torch.zeros((2, 128), dtype=torch.bfloat16), None, None, 1, None, None)
    with pytest.raises(TypeError):
        i8h.moe_down_mxfp4_combine(torch.zeros((2, 32), dtype=torch.float16), None, None, {})
    with pytest.raises(TypeError):
        i8h.draft_verify(torch.zeros((1, 2, 3), dtype=torch.float64), None, None, None, None)


def test_calls_run_on_their_tensors_device(monkeypatch):
    """Tensors of another device than the current one: the call makes theirs current and takes its stream."""
    current, seen = [0], []

    class Guard:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    class Lib:
        def draft_verify(self, *args):
            seen.append((current[0], args))
            return OK

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(i8h, "lib", lambda: Lib())
    i8h._call("draft_verify", torch.device("cuda", 0), 7)
    i8h._call("draft_verify", torch.device("cuda", 3), 8)
    assert seen == [(0, (7, 1000)), (3, (8, 1003))] and current == [0]


@pytest.fixture
def calls(monkeypatch):
    """The library's calls with their arguments, from tensors that hold no memory."""
    seen = []
    monkeypatch.setattr(i8h, "_dev", lambda t, *a, **kw: t)
    monkeypatch.setattr(i8h, "_call", lambda fn, device, *args: seen.append((fn, args)))
    return seen


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(32,), (5, 64), (2, 3, 64), ((1 << 31) - 32,), (1 << 31,), ((1 << 32) + 64,),
                                   (3, (1 << 32) + 32), (1 << 30, 32), (2, 1 << 33)])
def test_quantiser_takes_rows_of_any_length(calls, shape):
    """The library's sizes are 32-bit integers: what it is told has to cover the tensor, rows of 2^31 values too."""
    n = _meta(*shape).numel()
    codes, scales = i8h.mxfp4_quantize(_meta(*shape))
    assert codes.shape == shape[:-1] + (shape[-1] // 2,) and scales.shape == shape[:-1] + (shape[-1] // 32,)
    assert i8h.mxfp4_dequantize(codes, scales).shape == shape
    (q, (_, _, qt, qk, _, _)), (d, (_, _, dt, dk, _, _)) = calls
    assert q == "mxfp4_quantize" and d == "mxfp4_dequantize"
    for rows, K in ((qt, qk), (dt, dk)):
        assert rows * K == n and rows < 1 << 31 and K < 1 << 31 and K % 32 == 0


def test_quantiser_refuses_more_than_its_sizes_hold(calls):
    for shape in ((1 << 36,), (1 << 31, 32), (7, 1 << 34)):
        with pytest.raises(ValueError):
            i8h.mxfp4_quantize(_meta(*shape))
        with pytest.raises(ValueError):
            i8h.mxfp4_dequantize(_meta(*shape[:-1], shape[-1] // 2, dtype=torch.uint8),
                                 _meta(*shape[:-1], shape[-1] // 32, dtype=torch.uint8))
    assert not calls


@pytest.mark.parametrize("B,D,V", [(1, 0, (1 << 32) + 5), (1, 0, 1 << 31), ((1 << 32) + 1, 0, 1), (1 << 31, 0, 1),
                                   (1, (1 << 32) + 3, 1), (2, 1, (1 << 33) + 7)])
def test_draft_verify_refuses_sizes_past_32_bits(calls, B, D, V):
    """A size cut to 32 bits would be a smaller, valid one."""
    f, i = torch.float32, torch.int32
    with pytest.raises(ValueError):
        i8h.draft_verify(_meta(B, D + 1, V), None, _meta(B, D, dtype=i), _meta(B, D, dtype=f), _meta(B, dtype=f))
    assert not calls


def _meta_routing(T, E, topk):
    i = torch.int32
    return {"topk_ids": _meta(T, topk, dtype=i), "topk_w": _meta(T, topk, dtype=torch.float32),
            "expert_off": _meta(E + 1, dtype=i), "sorted_pairs": _meta(T * topk, dtype=i),
            "pair_pos": _meta(T * topk, dtype=i)}


@pytest.mark.parametrize("R,K", [(64, (1 << 32) + 128), (64, 1 << 32), (64, 1 << 31), ((1 << 32) + 64, 128),
                                 ((1 << 31) + 64, 128)])
def test_products_refuse_sizes_past_32_bits(L, calls, R, K):
    """Rows of the weights, and their number: cut to 32 bits they would be smaller, valid ones."""
    T, E, topk = 2, 3, 1
    codes, scales = _meta(E, R, K // 2, dtype=torch.uint8), _meta(E, R, K // 32, dtype=torch.uint8)
    r = _meta_routing(T, E, topk)
    with pytest.raises(ValueError):
        i8h.moe_gateup_mxfp4_grouped(_meta(T, K), codes, scales, topk, r["expert_off"], r["sorted_pairs"])
    with pytest.raises(ValueError):
        i8h.moe_down_mxfp4_combine(_meta(T * topk, K), codes, scales, r)
    assert not calls


@pytest.mark.parametrize("B", [1, 3])
def test_draft_workspace_of_the_largest_vocabularies(L, B):
    """Two float64 sums a chunk of 4096 entries and a count a sequence, up to V = 2^31 - 1."""
    for V in ((1 << 31) - 4096, (1 << 31) - 1024, (1 << 31) - 1023, (1 << 31) - 1):
        chunks = -(-V // 4096)
        assert L.draft_verify_workspace_size(B, V) == -(-(B * chunks * 16 + B * 4) // 256) * 256, V


def test_products_refuse_more_threads_than_a_launch_takes(L):
    """Rows past 8192 columns run as a workgroup per pass and 128 weight rows."""
    T, K, N = 493000, 8448, 508352
    need = L.moe_gateup_mxfp4_workspace_size(T, K, 1, 1)
    assert L.moe_gateup_mxfp4_grouped(A, T, K, A, A, 1, N, 1, A, A, None, A, 1, A, need, None) == EUNSUP
    need = L.moe_down_mxfp4_workspace_size(T, K, 1, N, 1)
    assert L.moe_down_mxfp4_combine(A, 1, T, K, A, A, 1, N, 1, A, A, A, A, A, A, need, None) == EUNSUP


@pytest.mark.parametrize("I", [8448, 1 << 27, 252645120, 252645120 + 256, 1 << 30, (1 << 31) - 256])
def test_workspace_of_the_longest_rows(L, I):
    """Rows past a workgroup's LDS: codes and scales padded to an odd number of 16-byte pieces, 16 bytes behind the
    last one, a list entry (16 bytes) for the head and at most each pass of 96 rows and expert, and y."""
    T, E, H, topk = 33, 4, 64, 1
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    row = (-(-17 * (I // 32) // 16) | 1) * 16
    assert L.moe_down_mxfp4_workspace_size(T, I, E, H, topk) == up(T * row + 16) + up(16 * (1 + T // 96 + E)) + up(T * H * 4)

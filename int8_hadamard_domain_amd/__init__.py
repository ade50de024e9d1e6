"""int8 Hadamard-domain MoE gate_up on AMD Instinct MI355X (gfx950).

Thin Python binding over libi8h.so (C ABI declared in include/i8h.h). Every
function here only checks tensors, allocates outputs with torch and passes
device pointers plus torch's current HIP stream to the library; all of the
computation runs in the library's HIP kernels. There is no CPU fallback: if
the library is not built, or a tensor is not on the GPU, the call raises.

Functions (same names as the C entry points):
  moe_route_permute          top-k routing and the expert-sorted permutation
  moe_route_permute_noalloc  the same without a workspace (fixed device scratch)
  moe_route_permute_rotate   routing plus the rotation of the routed tokens' rows
  hadamard128_rotate         blockwise 128-wide Walsh-Hadamard rotation (bf16)
  moe_gateup_i8h_grouped     grouped int8 Hadamard-domain gate_up + GELU epilogue
  moe_gateup_i8h_grouped_fused  the same on unrotated activations (rotation fused)
  moe_route_gateup_i8h_decode   routing + rotation + gate_up in one launch (few tokens)
  fp8_quantize_activations   per-token, per-128 E4M3 activation quantizer
  moe_gateup_fp8blk_grouped  grouped FP8 E4M3 128x128-block gate_up + epilogue
  moe_down_bf16_combine      bf16 grouped down projection + weighted combine
                             (the step after the path)
  linear_i8f16               dense int8 linear with f16 group scales (the
                             drafter's linears)
  i8_quantize_activations    per-token, per-128 int8 activation quantizer (W8A8)
  moe_gateup_i8g_grouped     grouped W8A8 int8 g128 gate_up + epilogue
  mxfp4_quantize             MXFP4 codes and scales of a matrix (blocks of 32)
  mxfp4_dequantize           the values that codes and scales stand for
  moe_gateup_mxfp4_grouped   grouped MXFP4 gate_up + epilogue
  moe_down_mxfp4_combine     grouped MXFP4 down projection + weighted combine
  draft_verify               which drafted tokens of a verify batch stay, and
                             the token sampled after them
  moe_route_scored_permute   routing by softmax or sigmoid scores, with a bias
                             for balance and groups of experts
  lora_add                   low-rank adapters of many requests beside any
                             projection's output
  linear_i8f16_lora          linear_i8f16 with the requests' adapters
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libi8h.so")

I8H_OK, I8H_EINVAL, I8H_EUNSUPPORTED, I8H_EHIP = 0, -1, -2, -3
PATHS = {"auto": 0, "gemv": 1, "gemm": 2, "tall": 3, "skinny": 4}
DOWN_PATHS = {"auto": 0, "gemv": 1, "gemm": 2}
TYPES = {torch.float32: 0, torch.bfloat16: 1}
SCORES = {"softmax": 0, "sigmoid": 1}
INT_MAX = (1 << 31) - 1   # the library's sizes are C ints, to which ctypes cuts a larger one without a word

_lib = None


class I8HError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = lib().i8h_status_string(status).decode()
        super().__init__(f"{fn} failed: {msg} ({status})")


def lib():
    """The loaded libi8h.so, with argument types set. Raises if not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                           "(python -m int8_hadamard_domain_amd.build_lib)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "i8h_status_string": (ctypes.c_char_p, [I]),
        "moe_route_permute_workspace_size": (SZ, [I, I, I]),
        "moe_route_permute": (I, [P, I, I, I, P, P, P, P, P, P, SZ, P]),
        "moe_route_permute_noalloc": (I, [P, I, I, I, P, P, P, P, P, P]),
        "moe_route_permute_rotate": (I, [P, P, I, I, I, I, P, P, P, P, P, P, P, SZ, P]),
        "hadamard128_rotate": (I, [P, I64, P, I64, I, I, P]),
        "moe_gateup_i8h_grouped": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P]),
        "moe_gateup_i8h_grouped_path": (I, [P, I, I, P, P, I, I, I, P, P, P, P, I, P]),
        "moe_gateup_i8h_grouped_act_bf16": (I, [P, I, I, P, P, I, I, I, P, P, P, P, I, P]),
        "moe_gateup_i8h_fused_workspace_size": (SZ, [I, I]),
        "moe_gateup_i8h_grouped_fused": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P, SZ, P]),
        "moe_route_gateup_i8h_decode": (I, [P, P, I, I, P, P, I, I, I, P, P, P, P, P, P, P, P]),
        "fp8_quantize_activations": (I, [P, I, I, P, P, P]),
        "moe_gateup_fp8blk_workspace_size": (SZ, [I, I]),
        "moe_gateup_fp8blk_grouped": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P, SZ, P]),
        "moe_gateup_fp8blk_grouped_path": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P, SZ, I, P]),
        "moe_gateup_fp8blk_grouped_act_bf16": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P, SZ, I, P]),
        "i8_quantize_activations": (I, [P, I, I, P, P, P]),
        "moe_gateup_i8g_workspace_size": (SZ, [I, I]),
        "moe_gateup_i8g_grouped": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P, SZ, P]),
        "moe_gateup_i8g_grouped_act_bf16": (I, [P, I, I, P, P, I, I, I, P, P, P, P, P, SZ, P]),
        "moe_down_bf16_workspace_size": (SZ, [I, I, I, I]),
        "moe_down_bf16_combine": (I, [P, I, I, P, I, I, I, P, P, P, P, P, P, SZ, P]),
        "moe_down_bf16_combine_path": (I, [P, I, I, P, I, I, I, P, P, P, P, P, P, SZ, I, P]),
        "moe_down_bf16_act_bf16_workspace_size": (SZ, [I, I, I, I]),
        "moe_down_bf16_combine_act_bf16": (I, [P, I, I, P, I, I, I, P, P, P, P, P, P, SZ, I, P]),
        "linear_i8f16": (I, [P, I, I, P, P, I, P, P]),
        "mxfp4_quantize": (I, [P, I, I, I, P, P, P]),
        "mxfp4_dequantize": (I, [P, P, I, I, P, I, P]),
        "moe_gateup_mxfp4_workspace_size": (SZ, [I, I, I, I]),
        "moe_gateup_mxfp4_grouped": (I, [P, I, I, P, P, I, I, I, P, P, P, P, I, P, SZ, P]),
        "moe_down_mxfp4_workspace_size": (SZ, [I, I, I, I, I]),
        "moe_down_mxfp4_combine": (I, [P, I, I, I, P, P, I, I, I, P, P, P, P, P, P, SZ, P]),
        "moe_route_scored_workspace_size": (SZ, [I, I, I]),
        "moe_route_scored_permute": (I, [P, I, I, I, I, I, P, I, I, I, I, F, P, P, P, P, P, P, SZ, P]),
        "lora_workspace_size": (SZ, [I, I]),
        "lora_add_workspace_size": (SZ, [I, I]),
        "lora_add": (I, [P, I, I64, P, I64, I, I, I, P, P, I, I, P, P, P, I64, P, SZ, P]),
        "linear_i8f16_lora": (I, [P, I, I, P, P, I, P, P, I, I, P, P, P, P, SZ, P]),
        "draft_verify_workspace_size": (SZ, [I, I]),
        "draft_verify": (I, [P, P, I, P, P, P, P, I, I, I, P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(fn, status):
    if status != I8H_OK:
        raise I8HError(fn, status)


def _dev(t, name, dtype, ndim=None, shape=None, device=None):
    """Check one tensor handed to the library: a torch.Tensor on the GPU (on
    `device` when given), of `dtype`, contiguous, with `ndim` dimensions or
    exactly `shape`. Raises TypeError / ValueError before anything is launched."""
    # the fitting tensor in one test (a call's checks are part of its latency);
    # the tests behind it only find what to say
    if type(t) is torch.Tensor and t.dtype is dtype and t.is_cuda and (shape is None or t.shape == shape) \
            and (ndim is None or t.dim() == ndim) and (device is None or t.device == device) and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions (got {t.dim()})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _workspace(ws, name, need, device):
    """A caller's byte workspace (uint8, 1-D, at least `need` bytes, on
    `device`), or a new one when ws is None."""
    if ws is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    _dev(ws, name, torch.uint8, 1, device=device)
    if ws.numel() < need:
        raise ValueError(f"{name} must hold at least {need} bytes (got {ws.numel()})")
    return ws


def _routing_outputs(out, T, E, topk, device):
    """The five routing tensors (from `out` where given, checked, else new)."""
    i32, f32 = torch.int32, torch.float32
    if not out:      # (the allocations are a third of a small call: sizes as plain numbers take 0.4 us less than tuples)
        pairs = torch.empty(T * topk, dtype=i32, device=device)
        return {"topk_ids": torch.empty((T, topk), dtype=i32, device=device),
                "topk_w": torch.empty((T, topk), dtype=f32, device=device),
                "expert_off": torch.empty(E + 1, dtype=i32, device=device),
                "sorted_pairs": pairs, "pair_pos": torch.empty_like(pairs)}
    o = dict(out)
    want = {"topk_ids": (i32, (T, topk)), "topk_w": (f32, (T, topk)), "expert_off": (i32, (E + 1,)),
            "sorted_pairs": (i32, (T * topk,)), "pair_pos": (i32, (T * topk,))}
    for key, (dt, shape) in want.items():
        if key in o:
            _dev(o[key], key, dt, shape=shape, device=device)
        else:
            o[key] = torch.empty(shape, dtype=dt, device=device)
    return o


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    # the handle itself: building torch.cuda.current_stream()'s Stream object takes 2 us a call
    return torch._C._cuda_getCurrentRawStream(device.index)


def moe_route_permute(logits, topk, out=None):
    """logits [T, E] float32 -> dict of topk_ids [T, k] int32, topk_w [T, k]
    float32, expert_off [E+1] int32, sorted_pairs [T*k] int32, pair_pos
    [T*k] int32 (and the workspace used). `out` may hold preallocated
    tensors under the same keys."""
    _dev(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    o = _routing_outputs(out, T, E, topk, dev)
    ws_bytes = lib().moe_route_permute_workspace_size(T, E, topk)
    o["workspace"] = _workspace(o.get("workspace"), "workspace", ws_bytes, dev)
    _check("moe_route_permute", lib().moe_route_permute(
        _ptr(logits), T, E, topk, _ptr(o["topk_ids"]), _ptr(o["topk_w"]), _ptr(o["expert_off"]),
        _ptr(o["sorted_pairs"]), _ptr(o["pair_pos"]), _ptr(o["workspace"]), o["workspace"].numel(),
        _stream(dev)))
    return o


def moe_route_permute_rotate(logits, x, topk, out=None, x_rot=None):
    """moe_route_permute on logits [T, E] float32, and the 128-wide Hadamard
    rotation of the activation rows x [T, K] bf16 in the same pass: returns
    the routing dict with "x_rot" [T, K] bf16 added (x_rot may be x itself)."""
    _dev(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    _dev(x, "x", torch.bfloat16, 2, device=dev)
    K = x.shape[1]
    _dev(x, "x", torch.bfloat16, shape=(T, K))
    o = _routing_outputs(out, T, E, topk, dev)
    xr = torch.empty_like(x) if x_rot is None else _dev(x_rot, "x_rot", torch.bfloat16, shape=(T, K), device=dev)
    ws_bytes = lib().moe_route_permute_workspace_size(T, E, topk)
    o["workspace"] = _workspace(o.get("workspace"), "workspace", ws_bytes, dev)
    _check("moe_route_permute_rotate", lib().moe_route_permute_rotate(
        _ptr(logits), _ptr(x), T, E, topk, K, _ptr(o["topk_ids"]), _ptr(o["topk_w"]), _ptr(o["expert_off"]),
        _ptr(o["sorted_pairs"]), _ptr(o["pair_pos"]), _ptr(xr), _ptr(o["workspace"]), o["workspace"].numel(),
        _stream(dev)))
    o["x_rot"] = xr
    return o


def moe_route_permute_noalloc(logits, topk, out=None):
    """moe_route_permute without a workspace: the library's own fixed device
    scratch holds the histograms (1 MiB per GPU; calls that overlap on one
    GPU race on it). Same results; `out` may hold the five output tensors."""
    _dev(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    o = _routing_outputs(out, T, E, topk, dev)
    _check("moe_route_permute_noalloc", lib().moe_route_permute_noalloc(
        _ptr(logits), T, E, topk, _ptr(o["topk_ids"]), _ptr(o["topk_w"]), _ptr(o["expert_off"]),
        _ptr(o["sorted_pairs"]), _ptr(o["pair_pos"]), _stream(dev)))
    return o


def hadamard128_rotate(x, out=None):
    """bf16 [T, K] (K % 128 == 0) -> bf16 [T, K], blockwise H x / sqrt(128).
    `out` may be x itself (in place)."""
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    y = torch.empty_like(x) if out is None else _dev(out, "out", torch.bfloat16, shape=(T, K), device=x.device)
    _check("hadamard128_rotate", lib().hadamard128_rotate(
        _ptr(x), K, _ptr(y), y.shape[1], T, K, _stream(x.device)))
    return y


def moe_gateup_i8h_grouped(x_rot, codes, scales, topk, expert_off, sorted_pairs,
                           gate_up=True, act=True, path="auto", act_dtype=torch.float32):
    """Grouped int8 Hadamard-domain gate_up.

    x_rot [T, K] bf16 (rotated), codes [E, N, K] int8, scales [E, N, K/128]
    bf16, expert_off [E+1] / sorted_pairs [T*topk] int32 from
    moe_route_permute. gate_up / act: True to allocate, a tensor to write
    into, or False/None to skip. act is float32, or bfloat16 (act_dtype, or
    the dtype of a given tensor: each value rounded to nearest even from the
    float32 one, the input moe_down_bf16_combine takes without rounding it
    again). Returns (gate_up, act) in expert-sorted row order (None for
    skipped outputs).
    """
    _dev(x_rot, "x_rot", torch.bfloat16, 2)
    T, K = x_rot.shape
    dev = x_rot.device
    _dev(codes, "codes", torch.int8, 3, device=dev)
    E, N, _ = codes.shape
    _dev(codes, "codes", torch.int8, shape=(E, N, K))
    _dev(scales, "scales", torch.bfloat16, shape=(E, N, K // 128), device=dev)
    _dev(expert_off, "expert_off", torch.int32, shape=(E + 1,), device=dev)
    _dev(sorted_pairs, "sorted_pairs", torch.int32, shape=(T * topk,), device=dev)
    gu = _out(gate_up, (T * topk, N), dev)
    adt = _act_dtype(act, act_dtype)
    ac = _out(act, (T * topk, N // 2), dev, adt)
    fn = "moe_gateup_i8h_grouped_act_bf16" if adt == torch.bfloat16 else "moe_gateup_i8h_grouped_path"
    _check(fn, getattr(lib(), fn)(
        _ptr(x_rot), T, K, _ptr(codes), _ptr(scales), E, N, topk, _ptr(expert_off), _ptr(sorted_pairs),
        _ptr(gu), _ptr(ac), PATHS[path], _stream(dev)))
    return gu, ac


def moe_gateup_i8h_grouped_fused(x, codes, scales, topk, expert_off, sorted_pairs,
                                 gate_up=True, act=True, workspace=None):
    """moe_gateup_i8h_grouped on UNROTATED bf16 activations x [T, K]: the
    128-wide Hadamard rotation is applied inside the call. Returns
    (gate_up, act)."""
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    _dev(codes, "codes", torch.int8, 3, device=dev)
    E, N, _ = codes.shape
    _dev(codes, "codes", torch.int8, shape=(E, N, K))
    _dev(scales, "scales", torch.bfloat16, shape=(E, N, K // 128), device=dev)
    _dev(expert_off, "expert_off", torch.int32, shape=(E + 1,), device=dev)
    _dev(sorted_pairs, "sorted_pairs", torch.int32, shape=(T * topk,), device=dev)
    need = lib().moe_gateup_i8h_fused_workspace_size(T, K)
    if need > 0 or workspace is not None:
        workspace = _workspace(workspace, "workspace", need, dev)
    gu = _out(gate_up, (T * topk, N), dev)
    ac = _out(act, (T * topk, N // 2), dev)
    _check("moe_gateup_i8h_grouped_fused", lib().moe_gateup_i8h_grouped_fused(
        _ptr(x), T, K, _ptr(codes), _ptr(scales), E, N, topk, _ptr(expert_off), _ptr(sorted_pairs),
        _ptr(gu), _ptr(ac), _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(dev)))
    return gu, ac


def moe_route_gateup_i8h_decode(logits, x, codes, scales, topk, gate_up=True, act=True, out=None):
    """Decode step in one launch: moe_route_permute on logits [T, E] float32,
    then the fused-rotation gate_up on UNROTATED x [T, K] bf16 (T*topk <= 64,
    E <= 256, K <= 4096). Returns (routing dict as moe_route_permute's,
    gate_up, act). `out` may hold preallocated routing tensors."""
    _dev(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    _dev(x, "x", torch.bfloat16, 2, device=dev)
    K = x.shape[1]
    _dev(x, "x", torch.bfloat16, shape=(T, K))
    _dev(codes, "codes", torch.int8, 3, device=dev)
    N = codes.shape[1]
    _dev(codes, "codes", torch.int8, shape=(E, N, K))
    _dev(scales, "scales", torch.bfloat16, shape=(E, N, K // 128), device=dev)
    o = _routing_outputs(out, T, E, topk, dev)
    gu = _out(gate_up, (T * topk, N), dev)
    ac = _out(act, (T * topk, N // 2), dev)
    _check("moe_route_gateup_i8h_decode", lib().moe_route_gateup_i8h_decode(
        _ptr(logits), _ptr(x), T, K, _ptr(codes), _ptr(scales), E, N, topk, _ptr(o["topk_ids"]),
        _ptr(o["topk_w"]), _ptr(o["expert_off"]), _ptr(o["sorted_pairs"]), _ptr(o["pair_pos"]),
        _ptr(gu), _ptr(ac), _stream(dev)))
    return o, gu, ac


def _out(spec, shape, dev, dtype=torch.float32):
    if spec is None or spec is False:
        return None
    if spec is True:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _dev(spec, "output", dtype, shape=shape, device=dev)


def _act_dtype(act, act_dtype):
    """The act output's dtype: a given tensor's own, else act_dtype (float32 or bfloat16)."""
    dt = act.dtype if isinstance(act, torch.Tensor) else act_dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"act must be float32 or bfloat16 (got {dt})")
    return dt


def fp8_quantize_activations(x, qx=None, sx=None):
    """bf16 [T, K] -> (E4M3 codes uint8 [T, K], float32 scales [T, K/128])."""
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    qx = (torch.empty((T, K), dtype=torch.uint8, device=dev) if qx is None
          else _dev(qx, "qx", torch.uint8, shape=(T, K), device=dev))
    sx = (torch.empty((T, K // 128), dtype=torch.float32, device=dev) if sx is None
          else _dev(sx, "sx", torch.float32, shape=(T, K // 128), device=dev))
    _check("fp8_quantize_activations", lib().fp8_quantize_activations(
        _ptr(x), T, K, _ptr(qx), _ptr(sx), _stream(x.device)))
    return qx, sx


def moe_gateup_fp8blk_grouped(x, codes, scales, topk, expert_off, sorted_pairs,
                              gate_up=True, act=True, workspace=None, path="auto", act_dtype=torch.float32):
    """Grouped FP8 E4M3 128x128-block gate_up.

    x [T, K] bf16 (not rotated), codes [E, N, K] uint8 (E4M3 bytes), scales
    [E, N/128, K/128] bf16. path: "auto", "gemm" or "skinny". act float32 or
    bfloat16 as for moe_gateup_i8h_grouped. Returns (gate_up, act,
    workspace); the workspace holds the quantized activations (see
    fp8_workspace_views).
    """
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    _dev(codes, "codes", torch.uint8, 3, device=dev)
    E, N, _ = codes.shape
    _dev(codes, "codes", torch.uint8, shape=(E, N, K))
    _dev(scales, "scales", torch.bfloat16, shape=(E, N // 128, K // 128), device=dev)
    _dev(expert_off, "expert_off", torch.int32, shape=(E + 1,), device=dev)
    _dev(sorted_pairs, "sorted_pairs", torch.int32, shape=(T * topk,), device=dev)
    need = lib().moe_gateup_fp8blk_workspace_size(T, K)
    workspace = _workspace(workspace, "workspace", need, dev)
    gu = _out(gate_up, (T * topk, N), dev)
    adt = _act_dtype(act, act_dtype)
    ac = _out(act, (T * topk, N // 2), dev, adt)
    fn = "moe_gateup_fp8blk_grouped_act_bf16" if adt == torch.bfloat16 else "moe_gateup_fp8blk_grouped_path"
    _check(fn, getattr(lib(), fn)(
        _ptr(x), T, K, _ptr(codes), _ptr(scales), E, N, topk, _ptr(expert_off), _ptr(sorted_pairs),
        _ptr(gu), _ptr(ac), _ptr(workspace), workspace.numel(), PATHS[path], _stream(dev)))
    return gu, ac, workspace


def fp8_workspace_views(workspace, T, K):
    """(qx [T, K] uint8, sx [T, K/128] float32, xq [T, K] bf16) views of a
    moe_gateup_fp8blk_grouped workspace: codes, scales and the codes' exact
    bf16 values."""
    up = lambda v: (v + 255) // 256 * 256
    a = up(T * K)
    b = a + up(T * (K // 128) * 4)
    qx = workspace[:T * K].view(T, K)
    sx = workspace[a:a + T * (K // 128) * 4].view(torch.float32).view(T, K // 128)
    xq = workspace[b:b + T * K * 2].view(torch.bfloat16).view(T, K)
    return qx, sx, xq


def moe_down_bf16_combine(act, w_down, routing, out=None, workspace=None, path="auto"):
    """bf16 grouped down projection of the expert-sorted act rows [P, I]
    float32 (rounded to bf16 for the product), or bfloat16 (taken as they
    are: the gate_up calls' bf16 act), against w_down [E, H, I] bf16, merged
    per token with the router weights: returns out [T, H] float32.
    `routing` is moe_route_permute's dict (topk_ids, topk_w, expert_off,
    pair_pos); `path` is "auto", "gemv" (one launch) or "gemm" (GEMM +
    combine)."""
    if not isinstance(act, torch.Tensor) or act.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("act must be a float32 or bfloat16 tensor")
    bf = act.dtype == torch.bfloat16
    _dev(act, "act", act.dtype, 2)
    P, I = act.shape
    dev = act.device
    _dev(w_down, "w_down", torch.bfloat16, 3, device=dev)
    E, H, _ = w_down.shape
    _dev(w_down, "w_down", torch.bfloat16, shape=(E, H, I))
    ids = _dev(routing["topk_ids"], "topk_ids", torch.int32, 2, device=dev)
    T, topk = ids.shape
    if P != T * topk:
        raise ValueError(f"act must have T * topk = {T * topk} rows (got {P})")
    tw = _dev(routing["topk_w"], "topk_w", torch.float32, shape=(T, topk), device=dev)
    off = _dev(routing["expert_off"], "expert_off", torch.int32, shape=(E + 1,), device=dev)
    pos = _dev(routing["pair_pos"], "pair_pos", torch.int32, shape=(P,), device=dev)
    need = (lib().moe_down_bf16_act_bf16_workspace_size if bf else lib().moe_down_bf16_workspace_size)(T, I, H, topk)
    if path != "gemv" or workspace is not None:
        workspace = _workspace(workspace, "workspace", need, dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _dev(out, "out", torch.float32, shape=(T, H), device=dev)
    fn = "moe_down_bf16_combine_act_bf16" if bf else "moe_down_bf16_combine_path"
    _check(fn, getattr(lib(), fn)(
        _ptr(act), T, I, _ptr(w_down), E, H, topk, _ptr(ids), _ptr(tw), _ptr(off), _ptr(pos), _ptr(out),
        _ptr(workspace), 0 if workspace is None else workspace.numel(), DOWN_PATHS[path], _stream(dev)))
    return out


def linear_i8f16(x, codes, scales, out=None):
    """Dense int8 linear: x [T, K] bf16 (unrotated), codes [N, K] int8,
    scales [N, K/128] float16 -> y [T, N] float32."""
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    _dev(codes, "codes", torch.int8, 2, device=dev)
    N = codes.shape[0]
    _dev(codes, "codes", torch.int8, shape=(N, K))
    _dev(scales, "scales", torch.float16, shape=(N, K // 128), device=dev)
    if out is None:
        out = torch.empty((T, N), dtype=torch.float32, device=dev)
    else:
        _dev(out, "out", torch.float32, shape=(T, N), device=dev)
    _check("linear_i8f16", lib().linear_i8f16(_ptr(x), T, K, _ptr(codes), _ptr(scales), N, _ptr(out), _stream(dev)))
    return out


def i8_quantize_activations(x):
    """x [T, K] bf16 -> (qx int8 [T, K], sx float32 [T, K/128])."""
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    qx = torch.empty((T, K), dtype=torch.int8, device=x.device)
    sx = torch.empty((T, K // 128), dtype=torch.float32, device=x.device)
    _check("i8_quantize_activations", lib().i8_quantize_activations(
        _ptr(x), T, K, _ptr(qx), _ptr(sx), _stream(x.device)))
    return qx, sx


def moe_gateup_i8g_grouped(x, codes, scales, topk, expert_off, sorted_pairs,
                           gate_up=True, act=True, workspace=None, act_dtype=torch.float32):
    """Grouped W8A8 int8 g128 gate_up.

    x [T, K] bf16 (not rotated), codes [E, N, K] int8, scales [E, N, K/128]
    bf16. act float32 or bfloat16 as for moe_gateup_i8h_grouped. Returns
    (gate_up, act, workspace); the workspace holds the int8 activations and
    their scales (see i8g_workspace_views).
    """
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    _dev(codes, "codes", torch.int8, 3, device=dev)
    E, N, _ = codes.shape
    _dev(codes, "codes", torch.int8, shape=(E, N, K))
    _dev(scales, "scales", torch.bfloat16, shape=(E, N, K // 128), device=dev)
    _dev(expert_off, "expert_off", torch.int32, shape=(E + 1,), device=dev)
    _dev(sorted_pairs, "sorted_pairs", torch.int32, shape=(T * topk,), device=dev)
    need = lib().moe_gateup_i8g_workspace_size(T, K)
    workspace = _workspace(workspace, "workspace", need, dev)
    gu = _out(gate_up, (T * topk, N), dev)
    adt = _act_dtype(act, act_dtype)
    ac = _out(act, (T * topk, N // 2), dev, adt)
    fn = "moe_gateup_i8g_grouped_act_bf16" if adt == torch.bfloat16 else "moe_gateup_i8g_grouped"
    _check(fn, getattr(lib(), fn)(
        _ptr(x), T, K, _ptr(codes), _ptr(scales), E, N, topk, _ptr(expert_off), _ptr(sorted_pairs),
        _ptr(gu), _ptr(ac), _ptr(workspace), workspace.numel(), _stream(dev)))
    return gu, ac, workspace


def i8g_workspace_views(workspace, T, K):
    """(qx [T, K] int8, sx [T, K/128] float32) views of a moe_gateup_i8g_grouped workspace."""
    a = (T * K + 255) // 256 * 256
    qx = workspace[:T * K].view(torch.int8).view(T, K)
    sx = workspace[a:a + T * (K // 128) * 4].view(torch.float32).view(T, K // 128)
    return qx, sx


def _call(fn, device, *args):
    """Call the library's fn(*args, stream) on `device`'s current stream, with
    `device` current: kernels launch on the current device only."""
    if torch._C._cuda_getDevice() != device.index:
        with torch.cuda.device(device):
            return _call(fn, device, *args)
    _check(fn, getattr(lib(), fn)(*args, _stream(device)))


def _type(t, name):
    """The library's element type of a float32 or bfloat16 tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in TYPES:
        raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
    return TYPES[t.dtype]


def _mx_weights(codes, scales, K, dev):
    """Check MXFP4 weights of K columns: codes [E, R, K/2], scales [E, R, K/32]. Returns (E, R)."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
        _dev(codes, "codes", torch.uint8, 3, device=dev)
    E, R, _ = codes.shape
    if K > INT_MAX or R > INT_MAX:
        raise ValueError(f"codes must have fewer than 2^31 rows and columns an expert (got {R} and {K})")
    _dev(codes, "codes", torch.uint8, shape=(E, R, K // 2), device=dev)
    _dev(scales, "scales", torch.uint8, shape=(E, R, K // 32), device=dev)
    return E, R


def _mx_out(t, name, shape, dtype, x):
    """A caller's tensor, checked, or a new one beside x."""
    if t is None:
        return x.new_empty(shape, dtype=dtype)
    return _dev(t, name, dtype, shape=shape, device=x.device)


def _mx_shape(t, name, unit, per_row):
    """(leading dimensions, last dimension, blocks of 32) of a matrix of whole blocks along its last dimension. Its
    rows lie one behind another, so the library takes it as so many rows of one block: its sizes are 32-bit."""
    shape = tuple(t.shape)
    if not shape or shape[-1] == 0 or shape[-1] % unit:
        raise ValueError(f"{name} must have a last dimension of whole blocks of {unit} (got {shape})")
    blocks = t.numel() // unit
    if blocks >= 1 << 31:
        raise ValueError(f"{name} must have fewer than 2^31 blocks (got {blocks})")
    return shape[:-1], shape[-1] * per_row, blocks


def mxfp4_quantize(x, codes=None, scales=None):
    """x [..., K] float32 or bfloat16 (K % 32 == 0) -> (codes uint8 [..., K/2],
    scales uint8 [..., K/32]): MXFP4, two E2M1 codes a byte (lower index in
    the low nibble) and an E8M0 scale per 32 values."""
    xt = _type(x, "x")
    _dev(x, "x", x.dtype)
    lead, K, blocks = _mx_shape(x, "x", 32, 1)
    codes = _mx_out(codes, "codes", lead + (K // 2,), torch.uint8, x)
    scales = _mx_out(scales, "scales", lead + (K // 32,), torch.uint8, x)
    _call("mxfp4_quantize", x.device, x.data_ptr(), xt, blocks, 32, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, out=None):
    """The values of MXFP4 codes [..., K/2] and scales [..., K/32] (uint8) as
    [..., K] float32 or bfloat16 (dtype, or the dtype of a given out)."""
    _dev(codes, "codes", torch.uint8)
    lead, K, blocks = _mx_shape(codes, "codes", 16, 2)
    _dev(scales, "scales", torch.uint8, shape=lead + (K // 32,), device=codes.device)
    if out is not None:
        dtype = out.dtype if isinstance(out, torch.Tensor) else None
    if dtype not in TYPES:
        raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
    out = _mx_out(out, "out", lead + (K,), dtype, codes)
    _call("mxfp4_dequantize", codes.device, codes.data_ptr(), scales.data_ptr(), blocks, 32, out.data_ptr(),
          TYPES[dtype])
    return out


def moe_gateup_mxfp4_grouped(x, codes, scales, topk, expert_off, sorted_pairs,
                             gate_up=True, act=True, workspace=None, act_dtype=torch.float32):
    """Grouped MXFP4 gate_up.

    x [T, K] bf16 (quantised to MXFP4 inside the call), codes [E, N, K/2]
    uint8, scales [E, N, K/32] uint8. gate_up, act and act_dtype as for
    moe_gateup_i8h_grouped. Returns (gate_up, act).
    """
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    E, N = _mx_weights(codes, scales, K, dev)
    _dev(expert_off, "expert_off", torch.int32, shape=(E + 1,), device=dev)
    _dev(sorted_pairs, "sorted_pairs", torch.int32, shape=(T * topk,), device=dev)
    need = lib().moe_gateup_mxfp4_workspace_size(T, K, E, topk)
    if need > 0 or workspace is not None:
        workspace = _workspace(workspace, "workspace", need, dev)
    gu = _out(gate_up, (T * topk, N), dev)
    adt = _act_dtype(act, act_dtype)
    ac = _out(act, (T * topk, N // 2), dev, adt)
    _call("moe_gateup_mxfp4_grouped", dev, _ptr(x), T, K, _ptr(codes), _ptr(scales), E, N, topk, _ptr(expert_off),
          _ptr(sorted_pairs), _ptr(gu), _ptr(ac), TYPES[adt], _ptr(workspace), need)
    return gu, ac


def moe_down_mxfp4_combine(act, codes, scales, routing, out=None, workspace=None):
    """MXFP4 grouped down projection of the expert-sorted act rows [P, I]
    (float32 or bfloat16, quantised inside the call) against codes [E, H, I/2]
    and scales [E, H, I/32] uint8, merged per token with the router weights:
    returns out [T, H] float32. `routing` is moe_route_permute's dict."""
    at = _type(act, "act")
    _dev(act, "act", act.dtype, 2)
    P, I = act.shape
    dev = act.device
    E, H = _mx_weights(codes, scales, I, dev)
    ids = _dev(routing["topk_ids"], "topk_ids", torch.int32, 2, device=dev)
    T, topk = ids.shape
    if P != T * topk:
        raise ValueError(f"act must have T * topk = {T * topk} rows (got {P})")
    tw = _dev(routing["topk_w"], "topk_w", torch.float32, shape=(T, topk), device=dev)
    off = _dev(routing["expert_off"], "expert_off", torch.int32, shape=(E + 1,), device=dev)
    pos = _dev(routing["pair_pos"], "pair_pos", torch.int32, shape=(P,), device=dev)
    need = lib().moe_down_mxfp4_workspace_size(T, I, E, H, topk)
    if need > 0 or workspace is not None:
        workspace = _workspace(workspace, "workspace", need, dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _dev(out, "out", torch.float32, shape=(T, H), device=dev)
    _call("moe_down_mxfp4_combine", dev, _ptr(act), at, T, I, _ptr(codes), _ptr(scales), E, H, topk, _ptr(ids),
          _ptr(tw), _ptr(off), _ptr(pos), _ptr(out), _ptr(workspace), need)
    return out


def draft_verify(target_probs, draft_probs, drafted, u, u_next, draft_len=None, tokens=None, accepted=None,
                 workspace=None):
    """Verification of drafted tokens (speculative sampling).

    target_probs [B, D+1, V], draft_probs [B, D, V] of the same type (float32
    or bfloat16), or None for tokens drafted without sampling; drafted [B, D]
    int32; u [B, D] and u_next [B] float32 uniform in [0, 1); draft_len [B]
    int32, or None for D everywhere. Returns (tokens [B, D+1] int32: the
    drafted tokens that stay, the token sampled after them, then -1; accepted
    [B] int32: how many stay).
    """
    pt = _type(target_probs, "target_probs")
    _dev(target_probs, "target_probs", target_probs.dtype, 3)
    B, D, V = target_probs.shape
    D -= 1
    dev = target_probs.device
    if D < 0:
        raise ValueError("target_probs must hold a row for each drafted token and one more")
    if B > INT_MAX or D > INT_MAX or V > INT_MAX:
        raise ValueError(f"target_probs must have dimensions below 2^31 (got {tuple(target_probs.shape)})")
    if draft_probs is not None:
        _dev(draft_probs, "draft_probs", target_probs.dtype, shape=(B, D, V), device=dev)
    _dev(drafted, "drafted", torch.int32, shape=(B, D), device=dev)
    _dev(u, "u", torch.float32, shape=(B, D), device=dev)
    _dev(u_next, "u_next", torch.float32, shape=(B,), device=dev)
    if draft_len is not None:
        _dev(draft_len, "draft_len", torch.int32, shape=(B,), device=dev)
    tokens = (drafted.new_empty((B, D + 1)) if tokens is None
              else _dev(tokens, "tokens", torch.int32, shape=(B, D + 1), device=dev))
    accepted = (drafted.new_empty(B) if accepted is None
                else _dev(accepted, "accepted", torch.int32, shape=(B,), device=dev))
    workspace = _workspace(workspace, "workspace", lib().draft_verify_workspace_size(B, V), dev)
    _call("draft_verify", dev, _ptr(target_probs), _ptr(draft_probs), pt, _ptr(drafted), _ptr(draft_len), _ptr(u),
          _ptr(u_next), B, D, V, _ptr(tokens), _ptr(accepted), _ptr(workspace), workspace.numel())
    return tokens, accepted


def moe_route_scored_permute(logits, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1,
                             renormalize=True, scale=1.0, out=None):
    """Routing by scores: logits [T, E] float32 or bfloat16 -> the dict of
    moe_route_permute.

    score: "softmax" (over all experts) or "sigmoid". The topk experts of
    largest score + bias (bias [E] float32, or None) are chosen, from the
    topk_groups of `groups` runs of experts whose group_top (1 or 2) largest
    values sum highest. topk_w holds their scores, divided by their sum with
    renormalize, times scale. `out` may hold preallocated tensors, the
    workspace among them.
    """
    lt = _type(logits, "logits")
    _dev(logits, "logits", logits.dtype, 2)
    T, E = logits.shape
    if T > INT_MAX or E > INT_MAX:
        raise ValueError(f"logits must have dimensions below 2^31 (got {tuple(logits.shape)})")
    dev = logits.device
    if score not in SCORES:
        raise ValueError(f'score must be "softmax" or "sigmoid" (got {score!r})')
    for name, v in (("topk", topk), ("groups", groups), ("topk_groups", topk_groups), ("group_top", group_top)):
        if not 0 < v <= INT_MAX:
            raise ValueError(f"{name} must be positive and below 2^31 (got {v})")
    if bias is not None:
        _dev(bias, "bias", torch.float32, shape=(E,), device=dev)
    o = _routing_outputs(out, T, E, topk, dev)
    need = lib().moe_route_scored_workspace_size(T, E, topk)
    if need > 0 or "workspace" in o:
        o["workspace"] = _workspace(o.get("workspace"), "workspace", need, dev)
    _call("moe_route_scored_permute", dev, _ptr(logits), lt, T, E, topk, SCORES[score], _ptr(bias), groups,
          topk_groups, group_top, 1 if renormalize else 0, scale, _ptr(o["topk_ids"]), _ptr(o["topk_w"]),
          _ptr(o["expert_off"]), _ptr(o["sorted_pairs"]), _ptr(o["pair_pos"]), _ptr(o.get("workspace")), need)
    return o


def _rows(t, name, dtype, shape, device):
    """Check a matrix of `dtype` whose rows are contiguous and may lie apart. Returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'the GPU'} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have {'2 dimensions' if shape is None else f'shape {tuple(shape)}'} "
                         f"(got {tuple(t.shape)})")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        return -(-cols // 8) * 8      # no second row: any distance will do
    if t.stride(0) < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.stride(0)


def _lora(lora_a, lora_b, adapter, lora_scale, T, K, N, dev):
    """Check the adapters [L, R, K] and [L, N, R] bf16, the rows' adapters [T] and the scales [L]. Returns (L, R)."""
    _dev(lora_a, "lora_a", torch.bfloat16, 3, device=dev)
    L, R, k = lora_a.shape
    if max(T, K, N, L, R) > INT_MAX:
        raise ValueError("sizes must be below 2^31")
    if k != K:
        _dev(lora_a, "lora_a", torch.bfloat16, shape=(L, R, K))
    _dev(lora_b, "lora_b", torch.bfloat16, shape=(L, N, R), device=dev)
    _dev(adapter, "adapter", torch.int32, shape=(T,), device=dev)
    _dev(lora_scale, "lora_scale", torch.float32, shape=(L,), device=dev)
    return L, R


def lora_add(base, x, lora_a, lora_b, adapter, lora_scale, out=None, workspace=None):
    """Low-rank adapters beside a projection: out[t] = base[t] + lora_scale[l]
    * lora_b[l] @ (lora_a[l] @ x[t]) with l = adapter[t]; rows whose adapter
    lies outside [0, L), for instance -1, are base's.

    base [T, N] float32 or bfloat16 (the projection's output), x [T, K] bf16
    (its input), lora_a [L, R, K] and lora_b [L, N, R] bf16, adapter [T]
    int32, lora_scale [L] float32. Rows of base, x and out may lie apart (a
    column slice of a wider matrix). `out` may be base. Returns out.
    """
    bt = _type(base, "base")
    ldb = _rows(base, "base", base.dtype, None, None)
    T, N = base.shape
    dev = base.device
    ldx = _rows(x, "x", torch.bfloat16, None, dev)
    if x.shape[0] != T:
        raise ValueError(f"x must have base's {T} rows (got {x.shape[0]})")
    K = x.shape[1]
    L, R = _lora(lora_a, lora_b, adapter, lora_scale, T, K, N, dev)
    if out is None:
        out = base.new_empty((T, N))
        ldo = N
    else:
        ldo = _rows(out, "out", base.dtype, base.shape, dev)
    need = lib().lora_add_workspace_size(T, R)
    if need > 0 or workspace is not None:
        workspace = _workspace(workspace, "workspace", need, dev)
    _call("lora_add", dev, _ptr(base), bt, ldb, _ptr(x), ldx, T, K, N, _ptr(lora_a), _ptr(lora_b), L, R,
          _ptr(adapter), _ptr(lora_scale), _ptr(out), ldo, _ptr(workspace), need)
    return out


def linear_i8f16_lora(x, codes, scales, lora_a, lora_b, adapter, lora_scale, out=None, workspace=None):
    """linear_i8f16 with the adapters of the rows' requests: x [T, K] bf16,
    codes [N, K] int8, scales [N, K/128] float16, adapters as for lora_add ->
    y [T, N] float32."""
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    _dev(codes, "codes", torch.int8, 2, device=dev)
    N, k = codes.shape
    L, R = _lora(lora_a, lora_b, adapter, lora_scale, T, K, N, dev)
    if k != K:
        _dev(codes, "codes", torch.int8, shape=(N, K))
    _dev(scales, "scales", torch.float16, shape=(N, K // 128), device=dev)
    if out is None:
        out = torch.empty((T, N), dtype=torch.float32, device=dev)
    else:
        _dev(out, "out", torch.float32, shape=(T, N), device=dev)
    workspace = _workspace(workspace, "workspace", lib().lora_workspace_size(T, R), dev)
    _call("linear_i8f16_lora", dev, _ptr(x), T, K, _ptr(codes), _ptr(scales), N, _ptr(lora_a), _ptr(lora_b), L, R,
          _ptr(adapter), _ptr(lora_scale), _ptr(out), _ptr(workspace), workspace.numel())
    return out

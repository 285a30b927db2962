"""Python binding of the library's C ABI (``include/moe.h``, ``include/moe_ops.h`` and
``include/moe_failures.h``), through ctypes.

Argument marshalling only: every step of the layer runs in the CUDA library ``libfp8moe.so``.
Importing this module loads that library and raises if it has not been built; there is no other
implementation to fall back to. Tensors are torch CUDA tensors (torch provides device memory and
streams); bf16 tensors are passed as their bit patterns and e4m3 tensors as uint8 codes.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8moe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_DEVICE_TIMEOUT = -5
MOE_ERR_DEVICE_CHECK = -6
NUM_STAGES = 8
STAGE_NAMES = ("router_logits", "topk_quant", "permute", "gather", "gemm_gateup_swiglu",
               "requant", "gemm_down", "combine")


class MoEDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("F", ctypes.c_int32), ("k_max", ctypes.c_int32), ("F_shared", ctypes.c_int32)]


class MoEDebugOut(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("expert_offsets", ctypes.c_void_p), ("perm_token", ctypes.c_void_p),
                ("inv_row", ctypes.c_void_p), ("y_f32", ctypes.c_void_p),
                ("stage_events", ctypes.POINTER(ctypes.c_void_p))]


class FFNDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("F", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32)]


# moe_dtype and moe_act of include/moe_ops.h
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTIVATIONS = {"silu": 0, "gelu": 1}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -m fp8_moe_layer_b200.build` "
            "(nvcc, sm_100a). The FP8 MoE layer has no other implementation.")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    dims_p = ctypes.POINTER(MoEDims)
    ffn_p = ctypes.POINTER(FFNDims)
    sig = {
        "moe_workspace_bytes": (sz, [dims_p]),
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_clear_status": (ctypes.c_int, [vp, vp]),
        "moe_device_status": (ctypes.c_int, [vp, vp, ctypes.POINTER(i32)]),
        "moe_route_topk": (ctypes.c_int, [dims_p, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]),
        "moe_permute": (ctypes.c_int, [dims_p, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
        "moe_grouped_ffn_fp8": (ctypes.c_int, [dims_p, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                               sz, vp]),
        "moe_combine": (ctypes.c_int, [dims_p, vp, vp, vp, vp, vp, vp, vp]),
        "moe_forward": (ctypes.c_int, [dims_p, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, sz, vp, ctypes.POINTER(MoEDebugOut)]),
        "moe_route_topk_noalloc": (ctypes.c_int, [dims_p, vp, vp, vp, i32, vp, vp, vp, vp]),
        "moe_device_failure": (ctypes.c_int, [i32, vp, vp]),
        "moe_kernel_launch_count": (ctypes.c_uint64, []),
        "moe_ep_dispatch": (ctypes.c_int, [dims_p, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                           vp, vp, sz, vp]),
        "moe_quant_int8": (ctypes.c_int, [ctypes.c_int64, i32, i32, vp, vp, vp, vp]),
        "moe_matmul_int8_workspace_bytes": (sz, [i32, i32, i32]),
        "moe_matmul_int8": (ctypes.c_int, [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp,
                                           vp, sz, vp]),
        "moe_grouped_ffn_int8": (ctypes.c_int, [dims_p, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                sz, vp]),
        "moe_gated_ffn_workspace_bytes": (sz, [ffn_p]),
        "moe_gated_ffn_backward_workspace_bytes": (sz, [ffn_p]),
        "moe_gated_ffn": (ctypes.c_int, [ffn_p, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_gated_ffn_backward": (ctypes.c_int, [ffn_p, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                                  vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def load_library(path: str) -> ctypes.CDLL:
    """Another build of the same C ABI (e.g. the wait-test build), with the argument types set."""
    return _load(path)


def kernel_launch_count() -> int:
    """Kernels the library has launched in this process so far (a host-side counter)."""
    return int(LIB.moe_kernel_launch_count())


def status_string(status: int) -> str:
    return LIB.moe_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def dims(T: int, d: int, E: int, F: int, k_max: int, F_shared: int = 0) -> MoEDims:
    return MoEDims(int(T), int(d), int(E), int(F), int(k_max), int(F_shared))


def workspace_bytes(dm: MoEDims) -> int:
    return int(LIB.moe_workspace_bytes(ctypes.byref(dm)))


def alloc_workspace(dm: MoEDims, device=None, also: Optional[MoEDims] = None) -> torch.Tensor:
    """Workspace for every entry point with these dims (and, one after the other, with those of
    ``also``), its status word cleared."""
    need = [workspace_bytes(m) for m in (dm, also) if m is not None]
    n = max(need)
    if min(need) == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    _check(LIB.moe_clear_status(ws.data_ptr(), _stream(ws.device)), "moe_clear_status")
    return ws


_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(device=None) -> int:
    """The current stream's handle (without building a torch Stream object around it)."""
    index = None if device is None else torch.device(device).index
    return _raw_stream(torch.cuda.current_device() if index is None else index)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _bits(t: torch.Tensor) -> torch.Tensor:
    """bf16 tensor -> its int16 view (bit patterns) without a copy."""
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16)
    if t.dtype in (torch.int16, torch.uint16):
        return t
    raise TypeError("expected a bf16 tensor")


def _u8(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError("expected e4m3 codes (uint8 or float8_e4m3fn)")
    return t


def device_status(ws: torch.Tensor) -> int:
    out = ctypes.c_int32(0)
    _check(LIB.moe_device_status(ws.data_ptr(), _stream(ws.device), ctypes.byref(out)),
           "moe_device_status")
    return int(out.value)


def clear_status(ws: torch.Tensor) -> None:
    _check(LIB.moe_clear_status(ws.data_ptr(), _stream(ws.device)), "moe_clear_status")


def device_failure(device=None, clear: bool = True) -> int:
    """The first failure that any kernel of the library recorded on ``device`` (default: the current
    one) since this was last asked, whichever workspace it went to: MOE_OK or a MOE_ERR_DEVICE_* code.

    A bounded wait that expired leaves its call's outputs incomplete. ``device_status`` says so for a
    workspace that its caller holds; this also covers the calls that take a workspace of their own
    (``ws=None``, ``gated_ffn`` and its backward pass, ``Int8GatedFFN``, replays of graphs). It waits
    for the current stream: ask once per step or batch, not per call, and not while capturing."""
    out = (ctypes.c_int32 * 3)()
    with torch.cuda.device(device):
        _check(LIB.moe_device_failure(int(clear), out, _stream()), "moe_device_failure")
    return int(out[0])


# ------------------------------------------------------------------------------ entry points
def moe_route_topk(hidden, router_w, router_bias, k, k_per_token, k_max, F=16, ws=None):
    """Router + softmax + top-k: returns (topk_ids int32 [T, k_max], topk_w fp32 [T, k_max])."""
    T, d = hidden.shape
    E = router_w.shape[0]
    dm = dims(T, d, E, F, k_max)
    ws = alloc_workspace(dm, hidden.device) if ws is None else ws
    ids = torch.empty(T, k_max, dtype=torch.int32, device=hidden.device)
    w = torch.empty(T, k_max, dtype=torch.float32, device=hidden.device)
    _check(LIB.moe_route_topk(ctypes.byref(dm), _p(_bits(hidden)), _p(router_w), _p(router_bias),
                              int(k), _p(k_per_token), _p(ids), _p(w), _p(ws), ws.numel(),
                              _stream(hidden.device)), "moe_route_topk")
    return ids, w


def moe_permute(topk_ids, k, k_per_token, E, d=16, F=16, ws=None):
    """Stable grouping by expert: returns (expert_offsets [E+1], perm_token [T*k_max],
    inv_row [T, k_max]), all int32."""
    T, k_max = topk_ids.shape
    dm = dims(T, d, E, F, k_max)
    ws = alloc_workspace(dm, topk_ids.device) if ws is None else ws
    dev = topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.full((max(T * k_max, 1),), -1, dtype=torch.int32, device=dev)
    inv = torch.empty(T, k_max, dtype=torch.int32, device=dev)
    _check(LIB.moe_permute(ctypes.byref(dm), _p(topk_ids), int(k), _p(k_per_token), _p(offsets),
                           _p(perm), _p(inv), _p(ws), ws.numel(), _stream(dev)), "moe_permute")
    return offsets, perm, inv


def moe_grouped_ffn_fp8(hidden, w13, w13_scale, w2, w2_scale, expert_offsets, perm_token, k_max,
                        ws=None, want_act_scale=False):
    """Grouped W8A8 FP8 SwiGLU experts over routed rows: returns expert_out fp32 [T*k_max, d]
    (and the per-token activation scales when asked)."""
    T, d = hidden.shape
    E, twoF, _ = w13.shape
    dm = dims(T, d, E, twoF // 2, k_max)
    dev = hidden.device
    ws = alloc_workspace(dm, dev) if ws is None else ws
    out = torch.zeros(max(T * k_max, 1), d, dtype=torch.float32, device=dev)
    xs = torch.empty(T, dtype=torch.float32, device=dev) if want_act_scale else None
    _check(LIB.moe_grouped_ffn_fp8(ctypes.byref(dm), _p(_bits(hidden)), _p(_u8(w13)),
                                   _p(w13_scale), _p(_u8(w2)), _p(w2_scale), _p(expert_offsets),
                                   _p(perm_token), _p(out), _p(xs), _p(ws), ws.numel(),
                                   _stream(dev)), "moe_grouped_ffn_fp8")
    return (out, xs) if want_act_scale else out


def moe_grouped_ffn_int8(hidden, w13, w13_scale, w2, w2_scale, expert_offsets, perm_token, k_max,
                         ws=None, want_act_scale=False):
    """Grouped W8A8 int8 SwiGLU experts over routed rows: ``moe_grouped_ffn_fp8`` with int8 codes
    (w13 [E, 2F, d], w2 [E, d, F], scales as there). Returns expert_out fp32 [T*k_max, d] (rows
    behind the last routed one are zero), and the per-token activation scales when asked."""
    if hidden.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("hidden must be [T, d], w13 [E, 2F, d] and w2 [E, d, F]")
    T, d = hidden.shape
    E, F, dev = w13.shape[0], w2.shape[2], hidden.device
    dm = dims(T, d, E, F, k_max)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return moe_grouped_ffn_int8(hidden, w13, w13_scale, w2, w2_scale, expert_offsets,
                                        perm_token, k_max, ws, want_act_scale)
    args = [_arg("hidden", hidden, torch.bfloat16, (T, d), dev),
            _arg("w13", w13, torch.int8, (E, 2 * F, d), dev),
            _arg("w13_scale", w13_scale, torch.float32, (E, 2 * F), dev),
            _arg("w2", w2, torch.int8, (E, d, F), dev),
            _arg("w2_scale", w2_scale, torch.float32, (E, d), dev),
            _arg("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev)]
    if perm_token.dtype != torch.int32 or perm_token.device != dev:
        raise TypeError(f"perm_token must be int32 on {dev}")
    if perm_token.numel() < T * k_max or not perm_token.is_contiguous():
        raise ValueError("perm_token must be contiguous and hold T * k_max rows")
    ws = alloc_workspace(dm, dev) if ws is None else _own_workspace(ws, dev)
    out = torch.empty(max(T * k_max, 1), d, dtype=torch.float32, device=dev)
    if T == 0:
        out.zero_()
    xs = torch.empty(T, dtype=torch.float32, device=dev) if want_act_scale else None
    _check(LIB.moe_grouped_ffn_int8(ctypes.byref(dm), *args, perm_token.data_ptr(),
                                    out.data_ptr(), _p(xs), _p(ws), ws.numel(),
                                    _raw_stream(dev.index)), "moe_grouped_ffn_int8")
    return (out, xs) if want_act_scale else out


def moe_combine(expert_out, topk_w, inv_row, shared_out=None, want_f32=False):
    """Weighted combine in token order: returns y bf16 [T, d] (and the fp32 sum when asked)."""
    T, k_max = topk_w.shape
    d = expert_out.shape[1]
    dm = dims(T, d, 1, 16, k_max)
    dev = expert_out.device
    y = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    yf = torch.empty(T, d, dtype=torch.float32, device=dev) if want_f32 else None
    _check(LIB.moe_combine(ctypes.byref(dm), _p(expert_out), _p(topk_w), _p(inv_row),
                           _p(shared_out), _p(y.view(torch.int16)), _p(yf), _stream(dev)),
           "moe_combine")
    return (y, yf) if want_f32 else y


def ep_local_k(E: int, k_max: int, n_ranks: int) -> int:
    """Expert slots per dispatched row: a token has at most min(k_max, E / n_ranks) experts on
    one rank."""
    return min(k_max, E // n_ranks)


def moe_ep_dispatch(hidden, topk_ids, topk_w, k, k_per_token, E, n_ranks, ws=None):
    """Expert-parallel dispatch plan and row gather. Returns a dict: send_hidden bf16
    [T*min(n_ranks, k_max), d], send_ids int32 / send_w fp32 [same rows, kl], send_counts int32
    [n_ranks] (device), slot_of int32 / slot_w fp32 [T, n_ranks]."""
    T, d = hidden.shape
    k_max = topk_ids.shape[1]
    dev = hidden.device
    dm = dims(T, d, E, 16, k_max)
    kl = ep_local_k(E, k_max, n_ranks)
    cap = max(T * min(n_ranks, k_max), 1)
    out = dict(send_hidden=torch.empty(cap, d, dtype=torch.bfloat16, device=dev),
               send_ids=torch.empty(cap, kl, dtype=torch.int32, device=dev),
               send_w=torch.empty(cap, kl, dtype=torch.float32, device=dev),
               send_counts=torch.empty(n_ranks, dtype=torch.int32, device=dev),
               slot_of=torch.empty(max(T, 1), n_ranks, dtype=torch.int32, device=dev),
               slot_w=torch.empty(max(T, 1), n_ranks, dtype=torch.float32, device=dev))
    ws = alloc_workspace(dims(max(T, 1), d, E, 16, k_max), dev) if ws is None else ws
    _check(LIB.moe_ep_dispatch(ctypes.byref(dm), int(n_ranks), _p(_bits(hidden)), _p(topk_ids),
                               _p(topk_w), int(k), _p(k_per_token),
                               _p(out["send_hidden"].view(torch.int16)), _p(out["send_ids"]),
                               _p(out["send_w"]), _p(out["send_counts"]), _p(out["slot_of"]),
                               _p(out["slot_w"]), _p(ws), ws.numel(), _stream(dev)),
           "moe_ep_dispatch")
    return out


def moe_forward(hidden, router_w, router_bias, k, k_per_token, w13, w13_scale, w2, w2_scale,
                k_max, shared: Optional[Sequence[torch.Tensor]] = None, ws=None, y=None,
                debug: bool = False, stage_events: Optional[Sequence] = None, lib=None):
    """The whole layer. Returns y bf16 [T, d], or (y, dict of debug outputs) when debug=True.
    ``lib``: another build of the library loaded with ``load_library`` (default: this one)."""
    T, d = hidden.shape
    E, twoF, _ = w13.shape
    F = twoF // 2
    Fs = shared[0].shape[0] // 2 if shared is not None else 0
    dm = dims(T, d, E, F, k_max, Fs)
    dev = hidden.device
    ws = alloc_workspace(dm, dev) if ws is None else ws
    y = torch.empty(T, d, dtype=torch.bfloat16, device=dev) if y is None else y
    w13s, s13s, w2s, s2s = shared if shared is not None else (None, None, None, None)
    dbg_struct, dbg = None, None
    ev_arr = None
    if debug or stage_events is not None:
        dbg = {}
        if debug:
            dbg = dict(topk_ids=torch.empty(T, k_max, dtype=torch.int32, device=dev),
                       topk_w=torch.empty(T, k_max, dtype=torch.float32, device=dev),
                       expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                       perm_token=torch.empty(max(T * k_max, 1), dtype=torch.int32, device=dev),
                       inv_row=torch.empty(T, k_max, dtype=torch.int32, device=dev),
                       y_f32=torch.empty(T, d, dtype=torch.float32, device=dev))
        if stage_events is not None:
            for e in stage_events:            # torch creates its events lazily, on first record
                if e is not None and not e.cuda_event:
                    e.record()
            ev_arr = (ctypes.c_void_p * (NUM_STAGES + 1))(
                *[ctypes.c_void_p(e.cuda_event if e is not None else 0) for e in stage_events])
        dbg_struct = MoEDebugOut(*(dbg[n].data_ptr() if n in dbg else None for n in
                                   ("topk_ids", "topk_w", "expert_offsets", "perm_token",
                                    "inv_row", "y_f32")),
                                 ctypes.cast(ev_arr, ctypes.POINTER(ctypes.c_void_p))
                                 if ev_arr is not None else None)
    status = (lib or LIB).moe_forward(
        ctypes.byref(dm), _p(_bits(hidden)), _p(router_w), _p(router_bias), int(k),
        _p(k_per_token), _p(_u8(w13)), _p(w13_scale), _p(_u8(w2)), _p(w2_scale), _p(_u8(w13s)),
        _p(s13s), _p(_u8(w2s)), _p(s2s), _p(y.view(torch.int16)), _p(ws), ws.numel(),
        _stream(dev), ctypes.byref(dbg_struct) if dbg_struct is not None else None)
    _check(status, "moe_forward")
    return (y, dbg) if debug else y


# ------------------------------------------------------------------ int8 and 16-bit operators
def _elsewhere(device: torch.device) -> bool:
    """Whether the tensors' device is not the current one. The library launches on the current
    device, so the caller then makes theirs current and calls again."""
    if device.type != "cuda":
        raise ValueError("tensor must be on a CUDA device")
    return device.index != torch.cuda.current_device()


def _arg(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """Pointer of a contiguous, 16-byte aligned tensor of this dtype, shape and device."""
    p = t.data_ptr()
    if (t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()
            and not p & 15):
        return p
    _expect(name, t, dtype, shape, device)
    raise ValueError(f"{name} must be contiguous" if not t.is_contiguous()
                     else f"{name} must be 16-byte aligned")


def _expect(name: str, t: torch.Tensor, dtype, shape, device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")


def _no_derivative(where: str, x: torch.Tensor) -> None:
    """Refuses an input whose derivative is wanted: a result without a graph would pass for one that
    does not depend on it."""
    if x.requires_grad and torch.is_grad_enabled():
        raise RuntimeError(f"{where} has no backward pass: detach its input, or call it under "
                           "torch.no_grad()")
    if forward_ad.unpack_dual(x).tangent is not None:
        raise NotImplementedError(f"{where} has no forward-mode derivative")


def _workspace(ws: Optional[torch.Tensor], need: int, where: str, device) -> torch.Tensor:
    """The caller's workspace, or one from torch's allocator (reused in stream order)."""
    if need == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, where)
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    return _own_workspace(ws, device)


def _own_workspace(ws: torch.Tensor, device) -> torch.Tensor:
    """A caller's workspace, whose elements have to be its bytes (an expanded one has fewer)."""
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {device}")
    return ws


def moe_quant_int8(x):
    """Symmetric int8 quantisation of the rows of x [..., K] (bf16, fp16 or fp32; K a multiple of
    16): returns (codes int8 [..., K], scale fp32 [...])."""
    if x.dtype not in DTYPES:
        raise TypeError("x must be bf16, fp16 or fp32")
    if x.dim() < 1:
        raise ValueError("x must have a last dimension")
    K, dev = x.shape[-1], x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return moe_quant_int8(x)
    codes = torch.empty(x.shape, dtype=torch.int8, device=dev)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    _check(LIB.moe_quant_int8(scale.numel(), K, DTYPES[x.dtype],
                              _arg("x", x, x.dtype, x.shape, dev), codes.data_ptr(),
                              scale.data_ptr(), _raw_stream(dev.index)), "moe_quant_int8")
    return codes, scale


def moe_matmul_int8(x, w, w_scale, bias=None, x_scale=None, out_dtype=None, ws=None):
    """W8A8 product with a scale per token and output channel: [T, K] x [N, K] -> [T, N].

    x is bf16, fp16 or fp32 (each token is quantised here) or int8 codes with ``x_scale`` fp32 [T];
    w int8 [N, K]; w_scale fp32 [N]; bias fp32 [N] or None. ``out_dtype`` defaults to x's dtype, or
    bf16 for codes. K and N are multiples of 16."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [T, K] and w [N, K]")
    T, K = x.shape
    N, dev = w.shape[0], x.device
    codes = x.dtype == torch.int8
    if not codes and x.dtype not in DTYPES:
        raise TypeError("x must be bf16, fp16, fp32 or int8 codes")
    if codes != (x_scale is not None):
        raise ValueError("x_scale goes with int8 codes, and only with them")
    out_dtype = out_dtype or (torch.bfloat16 if codes else x.dtype)
    if out_dtype not in DTYPES:
        raise TypeError("out_dtype must be bf16, fp16 or fp32")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return moe_matmul_int8(x, w, w_scale, bias, x_scale, out_dtype, ws)
    xp = _arg("x", x, x.dtype, x.shape, dev)
    wp = _arg("w", w, torch.int8, (N, K), dev)
    sp = _arg("w_scale", w_scale, torch.float32, (N,), dev)
    bp = None if bias is None else _arg("bias", bias, torch.float32, (N,), dev)
    xs = _arg("x_scale", x_scale, torch.float32, (T,), dev) if codes else None
    ws = _workspace(ws, LIB.moe_matmul_int8_workspace_bytes(T, N, K), "moe_matmul_int8", dev)
    out = torch.empty(T, N, dtype=out_dtype, device=dev)
    _check(LIB.moe_matmul_int8(T, N, K, DTYPES.get(x.dtype, 0), None if codes else xp,
                               xp if codes else None, xs, wp, sp, bp, DTYPES[out_dtype],
                               out.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev.index)),
           "moe_matmul_int8")
    return out


def _ffn_dims(x, w13, w2, activation) -> FFNDims:
    if x.dim() != 2 or w13.dim() != 2 or w2.dim() != 2:
        raise ValueError("x must be [T, d], w13 [2F, d] and w2 [d, F]")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("the gated FFN takes bf16 or fp16")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return FFNDims(x.shape[0], x.shape[1], w2.shape[1], DTYPES[x.dtype], ACTIVATIONS[activation])


def moe_gated_ffn(x, w13, w2, activation="silu", save_h=False, ws=None):
    """y = (act(x Wg^T) * (x Wu^T)) W2^T in bf16 or fp16: x [T, d], w13 [2F, d] (gate rows, then up
    rows), w2 [d, F]; ``activation`` "silu" or "gelu" (tanh form). Returns y [T, d], and with
    ``save_h`` also h [T, 2F], the pre-activations that the backward pass takes."""
    dm = _ffn_dims(x, w13, w2, activation)
    T, d, F, dev, dt = dm.T, dm.d, dm.F, x.device, x.dtype
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return moe_gated_ffn(x, w13, w2, activation, save_h, ws)
    xp, w13p = _arg("x", x, dt, (T, d), dev), _arg("w13", w13, dt, (2 * F, d), dev)
    w2p = _arg("w2", w2, dt, (d, F), dev)
    ws = _workspace(ws, LIB.moe_gated_ffn_workspace_bytes(ctypes.byref(dm)), "moe_gated_ffn",
                    dev)
    y = torch.empty(T, d, dtype=dt, device=dev)
    h = torch.empty(T, 2 * F, dtype=dt, device=dev) if save_h else None
    _check(LIB.moe_gated_ffn(ctypes.byref(dm), xp, w13p, w2p, y.data_ptr(),
                             h.data_ptr() if save_h else None, ws.data_ptr(), ws.numel(),
                             _raw_stream(dev.index)), "moe_gated_ffn")
    return (y, h) if save_h else y


def moe_gated_ffn_backward(dy, x, w13, w2, h, activation="silu", need=(True, True, True), ws=None):
    """Gradients (dx [T, d], dw13 [2F, d], dw2 [d, F]) of ``moe_gated_ffn`` for dy [T, d], at the h
    that the forward call kept. ``need`` says which are wanted; the others come back as None."""
    dm = _ffn_dims(x, w13, w2, activation)
    T, d, F, dev, dt = dm.T, dm.d, dm.F, x.device, x.dtype
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return moe_gated_ffn_backward(dy, x, w13, w2, h, activation, need, ws)
    dyp, xp = _arg("dy", dy, dt, (T, d), dev), _arg("x", x, dt, (T, d), dev)
    w13p, w2p = _arg("w13", w13, dt, (2 * F, d), dev), _arg("w2", w2, dt, (d, F), dev)
    hp = _arg("h", h, dt, (T, 2 * F), dev)
    ws = _workspace(ws, LIB.moe_gated_ffn_backward_workspace_bytes(ctypes.byref(dm)),
                    "moe_gated_ffn_backward", dev)
    grads = tuple(torch.empty(n, dtype=dt, device=dev) if want else None
                  for n, want in zip(((T, d), (2 * F, d), (d, F)), need))
    gp = [None if g is None else g.data_ptr() for g in grads]
    _check(LIB.moe_gated_ffn_backward(ctypes.byref(dm), dyp, xp, w13p, w2p, hp, *gp,
                                      ws.data_ptr(), ws.numel(), _raw_stream(dev.index)),
           "moe_gated_ffn_backward")
    return grads


class MoELayerFP8:
    """Device-resident FP8 MoE layer: owns the weights and a workspace sized for ``max_T``."""

    def __init__(self, inputs, device="cuda", max_T: Optional[int] = None):
        s = inputs.shape
        self.shape = s
        self.device = torch.device(device)
        dev = self.device
        self.router_w = inputs.router_w.to(dev)
        self.router_bias = None if inputs.router_bias is None else inputs.router_bias.to(dev)
        self.w13, self.w13_scale = inputs.w13.to(dev), inputs.w13_scale.to(dev)
        self.w2, self.w2_scale = inputs.w2.to(dev), inputs.w2_scale.to(dev)
        self.shared = None
        if s.F_shared:
            self.shared = (inputs.w13_shared.to(dev), inputs.w13s_scale.to(dev),
                           inputs.w2_shared.to(dev), inputs.w2s_scale.to(dev))
        self.max_T = max_T or s.T
        self.dims = dims(self.max_T, s.d, s.E, s.F, s.k_max, s.F_shared)
        # split counts depend on T, so size the workspace for the largest need over 1..max_T
        need = max(workspace_bytes(dims(t, s.d, s.E, s.F, s.k_max, s.F_shared))
                   for t in range(1, self.max_T + 1))
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        clear_status(self.ws)

    def __call__(self, hidden, k_per_token=None, y=None, debug=False, stage_events=None,
                 k: Optional[int] = None):
        """y = layer(hidden); per-token k from ``k_per_token`` if given, else the fixed ``k``
        (default: the layer's k)."""
        if hidden.shape[0] > self.max_T:
            raise ValueError("more tokens than the workspace was sized for")
        k = self.shape.k if k is None else int(k)
        return moe_forward(hidden, self.router_w, self.router_bias, k, k_per_token,
                           self.w13, self.w13_scale, self.w2, self.w2_scale, self.shape.k_max,
                           shared=self.shared, ws=self.ws, y=y, debug=debug,
                           stage_events=stage_events)


class MoELayerInt8:
    """Device-resident MoE layer with W8A8 int8 experts: ``MoELayerFP8`` with int8 codes in place of
    e4m3, run through the split entry points (route, permute, grouped int8 FFN, combine).

    router_w [E, d] and router_bias [E] (or None) fp32; w13 [E, 2F, d], w2 [E, d, F] int8 with scales
    [E, 2F], [E, d]; shared = (w13 [2F, d], scale [2F], w2 [d, F], scale [d]) or None, an always-on
    expert of weight 1. The weights are constants, and hidden states whose gradient is wanted are
    refused. Each call takes its own workspace from torch's allocator, so calls of one layer
    may be captured or run on several streams; ``ws`` is the last call's (for ``device_status``)."""

    def __init__(self, router_w, router_bias, k, k_max, w13, w13_scale, w2, w2_scale, shared=None):
        if not 1 <= k <= k_max:
            raise ValueError("k must lie in [1, k_max]")
        if w2.dim() != 3:
            raise ValueError("w2 must be [E, d, F]")
        E, d, F = w2.shape
        _expect("router_w", router_w, torch.float32, (E, d), w2.device)
        if router_bias is not None:
            _expect("router_bias", router_bias, torch.float32, (E,), w2.device)
        _expect("w13", w13, torch.int8, (E, 2 * F, d), w2.device)
        self.router_w, self.router_bias = router_w, router_bias
        self.k, self.k_max = int(k), int(k_max)
        self.experts = (w13, w13_scale, w2, w2_scale)
        self.E, self.d, self.F = E, d, F
        self.shared = None if shared is None else tuple(t.unsqueeze(0) for t in shared)
        self.ws = None

    @classmethod
    def from_weights(cls, router_w, router_bias, k, k_max, w13, w2, shared=None):
        """The layer of bf16, fp16 or fp32 experts w13 [E, 2F, d], w2 [E, d, F] (and shared = (w13
        [2F, d], w2 [d, F])), one int8 scale per output channel."""
        if shared is not None:
            shared = (*moe_quant_int8(shared[0]), *moe_quant_int8(shared[1]))
        return cls(router_w, router_bias, k, k_max, *moe_quant_int8(w13), *moe_quant_int8(w2),
                   shared=shared)

    def __call__(self, hidden, k_per_token=None, k: Optional[int] = None):
        """y bf16 [T, d]; per-token k from ``k_per_token`` if given, else the fixed ``k``."""
        if hidden.dim() != 2:
            raise ValueError("hidden must be [T, d]")
        T, dev = hidden.shape[0], self.router_w.device
        _expect("hidden", hidden, torch.bfloat16, (T, self.d), dev)
        _no_derivative("MoELayerInt8", hidden)
        if k_per_token is not None:
            _expect("k_per_token", k_per_token, torch.int32, (T,), dev)
        k = self.k if k is None else int(k)
        if not 1 <= k <= self.k_max:
            raise ValueError("k must lie in [1, k_max]")
        if T == 0:
            return torch.empty_like(hidden)
        if _elsewhere(dev):
            with torch.cuda.device(dev):
                return self(hidden, k_per_token, k)
        # one workspace for the routed and the shared experts, so that its status word has the failures
        # of both; the last call's goes back to torch's allocator first
        also = None if self.shared is None else dims(T, self.d, 1, self.shared[2].shape[2], 1)
        self.ws = None
        self.ws = ws = alloc_workspace(dims(T, self.d, self.E, self.F, self.k_max), dev, also)
        ids, w = moe_route_topk(hidden, self.router_w, self.router_bias, k, k_per_token,
                                self.k_max, F=self.F, ws=ws)
        offsets, perm, inv = moe_permute(ids, k, k_per_token, self.E, d=self.d, F=self.F, ws=ws)
        out = moe_grouped_ffn_int8(hidden, *self.experts, offsets, perm, self.k_max, ws=ws)
        shared_out = None
        if self.shared is not None:
            one = torch.arange(2, dtype=torch.int32, device=dev) * T         # one expert's rows
            shared_out = moe_grouped_ffn_int8(
                hidden, *self.shared, one, torch.arange(T, dtype=torch.int32, device=dev), 1, ws=ws)
        return moe_combine(out, w, inv, shared_out=shared_out)

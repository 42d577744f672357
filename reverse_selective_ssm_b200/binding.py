"""ctypes binding of libr2l (include/r2l.h): argument marshalling only.

Every step of the layer runs in the CUDA library; this module turns torch
tensors into the raw device pointers and sizes the C ABI takes, calls it, and
raises :class:`R2LError` on a non-zero status.  There is no fallback: if the
shared library is missing or cannot be loaded, :func:`load` raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Optional, Sequence

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libr2l.so")

R2L_BF16, R2L_FP32 = 0, 1
R2L_FLAG_GENERAL_A = 0x1
R2L_FLAG_FORWARD_SCAN = 0x2
R2L_FLAG_SAVED_FORWARD = 0x4
R2L_FLAG_ACT8 = 0x8
R2L_DEVFLAG_LENGTH_CLAMPED = 0x1

STATUS = {0: "R2L_OK", 1: "R2L_ERR_INVALID_ARG", 2: "R2L_ERR_UNSUPPORTED", 3: "R2L_ERR_ALIGNMENT",
          4: "R2L_ERR_WORKSPACE", 5: "R2L_ERR_CUDA", 6: "R2L_ERR_DEVICE_CHECK"}

EXPORTS = ("r2l_abi_version", "r2l_status_string", "r2l_workspace_size", "r2l_sidecar_forward",
           "r2l_sidecar_forward_debug", "r2l_sidecar_forward_profiled", "r2l_sidecar_stack",
           "r2l_get_device_status", "r2l_reverse_scan_workspace_size", "r2l_reverse_scan",
           "r2l_reverse_scan_noalloc", "r2l_reverse_scan_backward_workspace_size",
           "r2l_reverse_scan_backward", "r2l_sidecar_backward_workspace_size", "r2l_sidecar_backward",
           "r2l_sidecar_forward_train", "r2l_gated_scan", "r2l_gated_scan_checkpoint_size",
           "r2l_gated_scan_train", "r2l_gated_scan_backward_workspace_size", "r2l_gated_scan_backward",
           "r2l_act8_pack", "r2l_act8_unpack")

NOALLOC_SCRATCH_BYTES = 16 << 20
GATED_TILE = 64      # positions between two states of a gated scan's checkpoint
ACT8_GROUP = 64      # channels that share a scale of an 8-bit activation checkpoint

STAGES = ("in_proj", "conv", "x_proj", "dt_proj", "scan", "out_proj", "ln_residual")


class R2LError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _LIB.r2l_status_string(status).decode() if _LIB is not None else STATUS.get(status, "?")
        super().__init__(f"{where}: {msg} (status {status})")


class Dims(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("d_inner", ctypes.c_int), ("d_state", ctypes.c_int),
                ("dt_rank", ctypes.c_int), ("d_conv", ctypes.c_int), ("dtype", ctypes.c_int),
                ("flags", ctypes.c_uint)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "in_proj_w", "conv_w", "conv_b", "x_proj_w", "dt_proj_w", "dt_proj_b", "A_log", "D",
        "out_proj_w", "ln_w", "ln_b")]


class Grads(ctypes.Structure):
    """r2l_grads: fp32 device arrays shaped like the weights."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "in_proj_w", "conv_w", "conv_b", "x_proj_w", "dt_proj_w", "dt_proj_b", "A_log", "D",
        "out_proj_w", "ln_w", "ln_b")]


class GatedIn(ctypes.Structure):
    """r2l_gated_in: x, r, g with their row strides, lam and h0."""
    _fields_ = [("x", ctypes.c_void_p), ("r", ctypes.c_void_p), ("g", ctypes.c_void_p), ("ldx", ctypes.c_int),
                ("ldr", ctypes.c_int), ("ldg", ctypes.c_int), ("lam", ctypes.c_void_p), ("h0", ctypes.c_void_p)]


class GatedGrads(ctypes.Structure):
    """r2l_gated_grads: dx, dr, dg with their row strides, dlam and dh0."""
    _fields_ = [("dx", ctypes.c_void_p), ("dr", ctypes.c_void_p), ("dg", ctypes.c_void_p), ("ld_dx", ctypes.c_int),
                ("ld_dr", ctypes.c_int), ("ld_dg", ctypes.c_int), ("dlam", ctypes.c_void_p),
                ("dh0", ctypes.c_void_p)]


class DebugOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "z", "u", "dbc", "y", "o", "hhat")]


_LIB: Optional[ctypes.CDLL] = None

# key of the synthetic weight dict -> field of the C struct
_WMAP = (("W_in", "in_proj_w"), ("conv_w", "conv_w"), ("conv_b", "conv_b"), ("W_x", "x_proj_w"),
         ("W_dt", "dt_proj_w"), ("b_dt", "dt_proj_b"), ("A_log", "A_log"), ("D", "D"),
         ("W_out", "out_proj_w"), ("ln_w", "ln_w"), ("ln_b", "ln_b"))


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libr2l.so (raises if it is missing: there is no other implementation)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libr2l.so not found at {path}; build it with "
                           "`python -m reverse_selective_ssm_b200.build`")
    lib = ctypes.CDLL(path)
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.r2l_abi_version.restype = ci
    lib.r2l_status_string.restype = ctypes.c_char_p
    lib.r2l_status_string.argtypes = [ci]
    lib.r2l_workspace_size.restype = ctypes.c_size_t
    lib.r2l_workspace_size.argtypes = [ctypes.POINTER(Dims), ci, ci]
    fwd = [vp, ctypes.POINTER(Weights), ctypes.POINTER(Dims), cf, ci, ci, vp, vp, ctypes.c_size_t, vp]
    lib.r2l_sidecar_forward.restype = ci
    lib.r2l_sidecar_forward.argtypes = fwd
    lib.r2l_sidecar_forward_debug.restype = ci
    lib.r2l_sidecar_forward_debug.argtypes = fwd + [ctypes.POINTER(DebugOut)]
    lib.r2l_sidecar_forward_profiled.restype = ci
    lib.r2l_sidecar_forward_profiled.argtypes = fwd + [ctypes.POINTER(vp), ci, ctypes.POINTER(ci)]
    lib.r2l_sidecar_stack.restype = ci
    lib.r2l_sidecar_stack.argtypes = [vp, ctypes.POINTER(Weights), ctypes.POINTER(cf), ci,
                                      ctypes.POINTER(Dims), ci, ci, vp, vp, ctypes.c_size_t, vp]
    lib.r2l_reverse_scan_workspace_size.restype = ctypes.c_size_t
    lib.r2l_reverse_scan_workspace_size.argtypes = [ctypes.POINTER(Dims), ci, ci, ci]
    lib.r2l_reverse_scan.restype = ci
    lib.r2l_reverse_scan.argtypes = [vp, vp, ci, vp, vp, ci, vp, vp, vp, vp, ctypes.POINTER(Dims), ci, ci, vp,
                                     ci, vp, ctypes.c_size_t, vp]
    lib.r2l_reverse_scan_noalloc.restype = ci
    lib.r2l_reverse_scan_noalloc.argtypes = [vp, vp, ci, vp, vp, ci, vp, vp, vp, vp, ctypes.POINTER(Dims), ci,
                                             ci, vp, ci, vp]
    lib.r2l_reverse_scan_backward_workspace_size.restype = ctypes.c_size_t
    lib.r2l_reverse_scan_backward_workspace_size.argtypes = [ctypes.POINTER(Dims), ci, ci, ci]
    lib.r2l_reverse_scan_backward.restype = ci
    lib.r2l_reverse_scan_backward.argtypes = [vp, vp, ci, vp, vp, ci, vp, vp, vp, vp, vp, vp, ci, vp, vp, ci,
                                              vp, vp, vp, ctypes.POINTER(Dims), ci, ci, vp, ci, vp,
                                              ctypes.c_size_t, vp]
    lib.r2l_sidecar_backward_workspace_size.restype = ctypes.c_size_t
    lib.r2l_sidecar_backward_workspace_size.argtypes = [ctypes.POINTER(Dims), ci, ci]
    lib.r2l_sidecar_backward.restype = ci
    lib.r2l_sidecar_backward.argtypes = [vp, ctypes.POINTER(Weights), ctypes.POINTER(Dims), cf, ci, ci, vp, vp, vp,
                                         vp, ctypes.POINTER(Grads), vp, ctypes.c_size_t, vp]
    lib.r2l_sidecar_forward_train.restype = ci
    lib.r2l_sidecar_forward_train.argtypes = [vp, vp, ctypes.POINTER(Weights), ctypes.POINTER(Dims), cf, ci, ci, vp,
                                              vp, ctypes.c_size_t, vp]
    gin, dp, sz = ctypes.POINTER(GatedIn), ctypes.POINTER(Dims), ctypes.c_size_t
    lib.r2l_gated_scan.restype = ci
    lib.r2l_gated_scan.argtypes = [gin, vp, ci, vp, dp, ci, ci, vp, vp, vp]
    lib.r2l_gated_scan_checkpoint_size.restype = sz
    lib.r2l_gated_scan_checkpoint_size.argtypes = [dp, ci, ci]
    lib.r2l_gated_scan_train.restype = ci
    lib.r2l_gated_scan_train.argtypes = [gin, vp, ci, vp, dp, ci, ci, vp, vp, sz, vp, vp]
    lib.r2l_gated_scan_backward_workspace_size.restype = sz
    lib.r2l_gated_scan_backward_workspace_size.argtypes = [dp, ci, ci]
    lib.r2l_gated_scan_backward.restype = ci
    lib.r2l_gated_scan_backward.argtypes = [gin, vp, ci, vp, ctypes.POINTER(GatedGrads), dp, ci, ci, vp, vp, sz, vp,
                                            sz, vp]
    lib.r2l_act8_pack.restype = ci
    lib.r2l_act8_pack.argtypes = [vp, ci, ci, ci, ci, ci, vp, vp, ci, vp, vp]
    lib.r2l_act8_unpack.restype = ci
    lib.r2l_act8_unpack.argtypes = [vp, ci, vp, ci, ci, ci, ci, vp, vp, ci, vp]
    lib.r2l_get_device_status.restype = ci
    lib.r2l_get_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
    _LIB = lib
    return lib


def make_dims(d_model: int, d_inner: int, d_state: int = 16, dt_rank: int = 128, d_conv: int = 4,
              dtype: torch.dtype = torch.bfloat16, flags: int = 0) -> Dims:
    code = {torch.bfloat16: R2L_BF16, torch.float32: R2L_FP32}[dtype]
    return Dims(d_model, d_inner, d_state, dt_rank, d_conv, code, flags)


def dims_of(dims, dtype: torch.dtype, flags: int = 0) -> Dims:
    """From a :class:`synthetic.Dims`-like object."""
    return make_dims(dims.d_model, dims.d_inner, dims.d_state, dims.dt_rank, dims.d_conv, dtype, flags)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libr2l takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libr2l takes contiguous tensors")
    return t.data_ptr()


def weights_struct(w: Dict[str, Optional[torch.Tensor]]) -> Weights:
    """Weights struct from a dict of device tensors (keys as in synthetic.WEIGHT_KEYS)."""
    ws = Weights()
    for key, field in _WMAP:
        setattr(ws, field, _ptr(w.get(key)))
    return ws


def workspace_size(dims: Dims, B: int, L: int) -> int:
    return int(load().r2l_workspace_size(ctypes.byref(dims), B, L))


def alloc_workspace(dims: Dims, B: int, L: int, device="cuda") -> torch.Tensor:
    n = workspace_size(dims, B, L)
    if n == 0:
        raise ValueError("invalid dims for a workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def sidecar_forward(hidden: torch.Tensor, weights, dims: Dims, s: float, lengths=None,
                    workspace: Optional[torch.Tensor] = None, stream=None, check: bool = True) -> int:
    """r2l_sidecar_forward on hidden [B, L, d] (in place)."""
    lib = load()
    B, L = hidden.shape[0], hidden.shape[1]
    if workspace is None:
        workspace = alloc_workspace(dims, B, L, hidden.device)
    w = weights if isinstance(weights, Weights) else weights_struct(weights)
    st = lib.r2l_sidecar_forward(_ptr(hidden), ctypes.byref(w), ctypes.byref(dims), float(s), B, L,
                                 _ptr(lengths), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_sidecar_forward")
    return st


def sidecar_forward_debug(hidden: torch.Tensor, weights, dims: Dims, s: float, lengths=None,
                          workspace: Optional[torch.Tensor] = None, stream=None,
                          outputs: Optional[Dict[str, torch.Tensor]] = None, check: bool = True) -> int:
    lib = load()
    B, L = hidden.shape[0], hidden.shape[1]
    if workspace is None:
        workspace = alloc_workspace(dims, B, L, hidden.device)
    w = weights if isinstance(weights, Weights) else weights_struct(weights)
    dbg = DebugOut()
    for k, v in (outputs or {}).items():
        setattr(dbg, k, _ptr(v))
    st = lib.r2l_sidecar_forward_debug(_ptr(hidden), ctypes.byref(w), ctypes.byref(dims), float(s), B, L,
                                       _ptr(lengths), _ptr(workspace), workspace.numel(),
                                       _stream_ptr(stream), ctypes.byref(dbg))
    if check and st != 0:
        raise R2LError(st, "r2l_sidecar_forward_debug")
    return st


def sidecar_forward_profiled(hidden: torch.Tensor, weights, dims: Dims, s: float, events, lengths=None,
                             workspace: Optional[torch.Tensor] = None, stream=None,
                             check: bool = True) -> int:
    """r2l_sidecar_forward_profiled: records ``events`` (len(STAGES)+1 torch
    CUDA events with timing) at the stage boundaries; returns the number of
    kernels the call enqueued."""
    lib = load()
    B, L = hidden.shape[0], hidden.shape[1]
    if workspace is None:
        workspace = alloc_workspace(dims, B, L, hidden.device)
    w = weights if isinstance(weights, Weights) else weights_struct(weights)
    for e in events:            # torch creates the CUDA event lazily on first record
        if not e.cuda_event:
            e.record(stream if stream is not None else torch.cuda.current_stream())
    ev = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    n = ctypes.c_int(0)
    st = lib.r2l_sidecar_forward_profiled(_ptr(hidden), ctypes.byref(w), ctypes.byref(dims), float(s), B, L,
                                          _ptr(lengths), _ptr(workspace), workspace.numel(),
                                          _stream_ptr(stream), ev, len(events), ctypes.byref(n))
    if check and st != 0:
        raise R2LError(st, "r2l_sidecar_forward_profiled")
    return int(n.value)


def sidecar_stack(hidden: torch.Tensor, weights_list: Sequence, dims: Dims, s_list: Sequence[float],
                  lengths=None, workspace: Optional[torch.Tensor] = None, stream=None,
                  check: bool = True) -> int:
    lib = load()
    B, L = hidden.shape[0], hidden.shape[1]
    if workspace is None:
        workspace = alloc_workspace(dims, B, L, hidden.device)
    n = len(weights_list)
    arr = (Weights * n)(*[w if isinstance(w, Weights) else weights_struct(w) for w in weights_list])
    sarr = (ctypes.c_float * n)(*[float(x) for x in s_list])
    st = lib.r2l_sidecar_stack(_ptr(hidden), arr, sarr, n, ctypes.byref(dims), B, L, _ptr(lengths),
                               _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_sidecar_stack")
    return st


def reverse_scan_workspace_size(dims: Dims, B: int, L: int, chunk_tokens: int = 0) -> int:
    return int(load().r2l_reverse_scan_workspace_size(ctypes.byref(dims), B, L, chunk_tokens))


def reverse_scan(u: torch.Tensor, z: torch.Tensor, dt_raw: torch.Tensor, bc: torch.Tensor,
                 A_log: torch.Tensor, D: torch.Tensor, dt_b: torch.Tensor, y: torch.Tensor, dims: Dims,
                 B: int, L: int, lengths=None, chunk_tokens: int = 0,
                 workspace: Optional[torch.Tensor] = None, stream=None, check: bool = True) -> int:
    """r2l_reverse_scan.  u, dt_raw, y: [B·L, E]; z: [B·L, ldz] (first E columns);
    bc: [B·L, ldbc] fp32 with B in columns 0..15 and C in 16..31."""
    lib = load()
    if workspace is None:
        n = reverse_scan_workspace_size(dims, B, L, chunk_tokens)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=u.device)
    st = lib.r2l_reverse_scan(_ptr(u), _ptr(z), z.stride(0), _ptr(dt_raw), _ptr(bc), bc.stride(0), _ptr(A_log),
                              _ptr(D), _ptr(dt_b), _ptr(y), ctypes.byref(dims), B, L, _ptr(lengths),
                              chunk_tokens, _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_reverse_scan")
    return st


def reverse_scan_noalloc(u: torch.Tensor, z: torch.Tensor, dt_raw: torch.Tensor, bc: torch.Tensor,
                         A_log: torch.Tensor, D: torch.Tensor, dt_b: torch.Tensor, y: torch.Tensor, dims: Dims,
                         B: int, L: int, lengths=None, chunk_tokens: int = 0, stream=None,
                         check: bool = True) -> int:
    """r2l_reverse_scan_noalloc: as :func:`reverse_scan`, with the library's
    static device scratch instead of a caller workspace (nothing is allocated)."""
    lib = load()
    st = lib.r2l_reverse_scan_noalloc(_ptr(u), _ptr(z), z.stride(0), _ptr(dt_raw), _ptr(bc), bc.stride(0),
                                      _ptr(A_log), _ptr(D), _ptr(dt_b), _ptr(y), ctypes.byref(dims), B, L,
                                      _ptr(lengths), chunk_tokens, _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_reverse_scan_noalloc")
    return st


def reverse_scan_backward_workspace_size(dims: Dims, B: int, L: int, chunk_tokens: int = 0) -> int:
    return int(load().r2l_reverse_scan_backward_workspace_size(ctypes.byref(dims), B, L, chunk_tokens))


def reverse_scan_backward(u: torch.Tensor, z: torch.Tensor, dt_raw: torch.Tensor, bc: torch.Tensor,
                          A_log: torch.Tensor, D: torch.Tensor, dt_b: torch.Tensor, dy: torch.Tensor,
                          du: torch.Tensor, dz: torch.Tensor, ddt_raw: torch.Tensor, dbc: torch.Tensor,
                          dA_log: torch.Tensor, dD: torch.Tensor, ddt_b: torch.Tensor, dims: Dims, B: int, L: int,
                          lengths=None, chunk_tokens: int = 0, workspace: Optional[torch.Tensor] = None,
                          stream=None, check: bool = True) -> int:
    """r2l_reverse_scan_backward (fp32).  u, dt_raw, dy, du, ddt_raw: [B·L, E];
    z, dz: [B·L, ld] (first E columns); bc, dbc: [B·L, ld] with B in columns
    0..15 and C in 16..31; dA_log [E, 16]; dD, ddt_b [E]."""
    lib = load()
    if workspace is None:
        n = reverse_scan_backward_workspace_size(dims, B, L, chunk_tokens)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=u.device)
    st = lib.r2l_reverse_scan_backward(_ptr(u), _ptr(z), z.stride(0), _ptr(dt_raw), _ptr(bc), bc.stride(0),
                                       _ptr(A_log), _ptr(D), _ptr(dt_b), _ptr(dy), _ptr(du), _ptr(dz), dz.stride(0),
                                       _ptr(ddt_raw), _ptr(dbc), dbc.stride(0), _ptr(dA_log), _ptr(dD),
                                       _ptr(ddt_b), ctypes.byref(dims), B, L, _ptr(lengths), chunk_tokens,
                                       _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_reverse_scan_backward")
    return st


def get_device_status(workspace: torch.Tensor, stream=None):
    """(status, flags) after synchronising the stream."""
    lib = load()
    flags = ctypes.c_uint32(0)
    st = lib.r2l_get_device_status(_ptr(workspace), _stream_ptr(stream), ctypes.byref(flags))
    return st, int(flags.value)


def weights_to_device(w: Dict[str, Optional[torch.Tensor]], device="cuda"):
    return {k: (None if v is None else v.to(device).contiguous()) for k, v in w.items()}


# weight-dict key -> r2l_grads field, as for the weights
GRAD_KEYS = tuple(k for k, _ in _WMAP)


def sidecar_backward_workspace_size(dims: Dims, B: int, L: int) -> int:
    return int(load().r2l_sidecar_backward_workspace_size(ctypes.byref(dims), B, L))


def alloc_grads(weights: Dict[str, Optional[torch.Tensor]], device="cuda") -> Dict[str, Optional[torch.Tensor]]:
    """fp32 gradient buffers shaped like a hook's weights (None where the
    weight is None)."""
    return {k: None if v is None else torch.empty(v.shape, dtype=torch.float32, device=device)
            for k, v in weights.items()}


def sidecar_forward_train(hidden: torch.Tensor, weights, dims: Dims, s: float, lengths=None,
                          workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None,
                          check: bool = True):
    """r2l_sidecar_forward_train: returns (out = h⁺, workspace); hidden is not
    written.  Pass the same workspace to sidecar_backward with dims carrying
    R2L_FLAG_SAVED_FORWARD to skip the forward's recomputation."""
    lib = load()
    B, L = hidden.shape[0], hidden.shape[1]
    if workspace is None:
        workspace = torch.empty(max(sidecar_backward_workspace_size(dims, B, L), 16), dtype=torch.uint8,
                                device=hidden.device)
    if out is None:
        out = torch.empty_like(hidden)
    w = weights if isinstance(weights, Weights) else weights_struct(weights)
    st = lib.r2l_sidecar_forward_train(_ptr(hidden), _ptr(out), ctypes.byref(w), ctypes.byref(dims), float(s), B, L,
                                       _ptr(lengths), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_sidecar_forward_train")
    return out, workspace


def sidecar_backward(hidden: torch.Tensor, weights, dims: Dims, s: float, dh_out: torch.Tensor,
                     grads: Dict[str, Optional[torch.Tensor]], lengths=None, workspace: Optional[torch.Tensor] = None,
                     stream=None, check: bool = True, dh: Optional[torch.Tensor] = None,
                     ds: Optional[torch.Tensor] = None):
    """r2l_sidecar_backward: returns (dh [B, L, d] fp32, ds (a 1-element fp32
    device tensor)); grads (from alloc_grads) receives every parameter's
    gradient.  dh and ds may be given (fp32 [B, L, d] and at least 4 floats,
    caller-owned); they are allocated here otherwise."""
    lib = load()
    B, L = hidden.shape[0], hidden.shape[1]
    if workspace is None:
        workspace = torch.empty(max(sidecar_backward_workspace_size(dims, B, L), 16), dtype=torch.uint8,
                                device=hidden.device)
    w = weights if isinstance(weights, Weights) else weights_struct(weights)
    g = Grads()
    for key, field in _WMAP:
        setattr(g, field, _ptr(grads.get(key)))
    if dh is None:
        dh = torch.empty(dh_out.shape, dtype=torch.float32, device=hidden.device)
    elif dh.dtype != torch.float32 or dh.shape != dh_out.shape:
        raise ValueError("dh must be fp32 and shaped like dh_out")
    if ds is None:
        ds = torch.zeros(4, dtype=torch.float32, device=hidden.device)
    elif ds.dtype != torch.float32 or ds.numel() < 4:
        raise ValueError("ds must be fp32 with at least 4 elements")
    st = lib.r2l_sidecar_backward(_ptr(hidden), ctypes.byref(w), ctypes.byref(dims), float(s), B, L, _ptr(lengths),
                                  _ptr(dh_out), _ptr(dh), _ptr(ds), ctypes.byref(g), _ptr(workspace),
                                  workspace.numel(), _stream_ptr(stream))
    if check and st != 0:
        raise R2LError(st, "r2l_sidecar_backward")
    return dh, ds[:1]


# ---------------------------------------------------------------- gated linear recurrence

_DTYPES = {R2L_BF16: torch.bfloat16, R2L_FP32: torch.float32}
_CODES = {v: k for k, v in _DTYPES.items()}


def gated_dims(channels: int, dtype: torch.dtype, flags: int = 0) -> Dims:
    """Dims of a gated scan over ``channels`` channels (the other fields are not read)."""
    return Dims(_int(channels), channels, 16, 1, 4, _CODES[dtype], flags)


def _int(v: int) -> int:
    """v, which the C interface takes as int (ctypes would pass its low 32 bits on)."""
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"sizes are below 2^31, got {v}")
    return v


def _positions(B: int, L: int) -> int:
    M = B * L
    if not 0 <= M < 1 << 31:         # else each is below 2^31, or one is 0, which the library refuses
        return _int(B) * _int(L)
    return M


@contextlib.contextmanager
def _elsewhere(device: torch.device, stream):
    """The device of a call's tensors made the current one, and its stream the one that its own tensors are allocated
    on (torch then reuses their memory in that stream's order); yields the raw stream."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            if not hasattr(stream, "cuda_stream"):
                # torch takes the handle 0 for a wish for a stream of its own
                raw = int(stream)
                stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _call_on(device: torch.device, stream, f):
    """f(raw stream) on this device and stream (None: the device's current one; a torch stream or a raw
    cudaStream_t).  Where the device is the current one and so is the stream, nothing is entered, and the raw stream is
    asked for directly: contexts and stream objects cost more than the launch of a decoding step."""
    if stream is None and device.index == torch.cuda.current_device():
        return f(torch._C._cuda_getCurrentRawStream(device.index))
    if getattr(stream, "device", device) != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with _elsewhere(device, stream) as st:
        return f(st)


def _rows(t: torch.Tensor, M: int, E: int, dtype: torch.dtype, device: torch.device, name: str):
    """(pointer, row stride) of [M, E] rows whose elements are contiguous: a tensor or columns of a wider one."""
    if t.shape != (M, E) or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} [{M}, {E}] on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    row, col = t.stride()
    if M == 1:          # a stride that leads nowhere
        row = E
    if (col != 1 and E > 1) or not E <= row < 1 << 31:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap, with a stride below 2^31 elements "
                         f"(strides {(row, col)})")
    return t.data_ptr(), row


def _vec(t: Optional[torch.Tensor], shape, device: torch.device, name: str,
         dtype: torch.dtype = torch.float32) -> Optional[int]:
    """Pointer of a contiguous tensor of this shape and type (None: null)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _bytes(t: torch.Tensor, device: torch.device, name: str):
    """(pointer, size in bytes) of a caller's buffer."""
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {device}, got {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _status(t: Optional[torch.Tensor], device: torch.device) -> Optional[int]:
    """Pointer of the device word that receives a call's status bits (None: not wanted)."""
    if t is None:
        return None
    p, size = _bytes(t, device, "status")
    if size < 4:
        raise ValueError(f"status must hold a word of 4 bytes, got {size}")
    return p


def _gated_inputs(x, r, g, lam, h0, dims, B, L):
    if not x.is_cuda:
        raise ValueError("libr2l takes device tensors")
    M, E, dtype, dev = _positions(B, L), dims.d_inner, _DTYPES[dims.dtype], x.device
    px, ldx = _rows(x, M, E, dtype, dev, "x")
    pr, ldr = _rows(r, M, E, dtype, dev, "r")
    pg, ldg = _rows(g, M, E, dtype, dev, "g")
    return GatedIn(px, pr, pg, ldx, ldr, ldg, _vec(lam, (E,), dev, "lam"), _vec(h0, (B, E), dev, "h0"))


def _gated_forward(x, r, g, lam, dims, B, L, h0, lengths, checkpoint, y, h_last, status, stream, check, train):
    lib = load()
    gi = _gated_inputs(x, r, g, lam, h0, dims, B, L)
    E, dev = dims.d_inner, x.device

    def call(st):
        nonlocal y, h_last, checkpoint
        if y is None:
            y = torch.empty((B * L, E), dtype=x.dtype, device=dev)
        if h_last is None:
            h_last = torch.empty((B, E), dtype=torch.float32, device=dev)
        py, ldy = _rows(y, B * L, E, x.dtype, dev, "y")
        ph = _vec(h_last, (B, E), dev, "h_last")
        pl = _vec(lengths, (B,), dev, "lengths", torch.int32)
        ps = None if status is None else _status(status, dev)
        if not train:
            return lib.r2l_gated_scan(gi, py, ldy, ph, dims, B, L, pl, ps, st)
        if checkpoint is None:
            checkpoint = torch.empty(lib.r2l_gated_scan_checkpoint_size(dims, B, L), dtype=torch.uint8, device=dev)
        return lib.r2l_gated_scan_train(gi, py, ldy, ph, dims, B, L, pl, *_bytes(checkpoint, dev, "checkpoint"), ps, st)

    rc = _call_on(dev, stream, call)
    if check and rc != 0:
        raise R2LError(rc, "r2l_gated_scan_train" if train else "r2l_gated_scan")
    return y, h_last, checkpoint


def gated_scan(x: torch.Tensor, r: torch.Tensor, g: torch.Tensor, lam: torch.Tensor, dims: Dims, B: int, L: int,
               h0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
               y: Optional[torch.Tensor] = None, h_last: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None, check: bool = True):
    """r2l_gated_scan: returns (y, h_last).  x, r, g, y: [B·L, E] rows of dims' dtype (columns of a wider tensor will
    do); lam fp32 [E]; h0, h_last fp32 [B, E] (h_last may be h0); lengths int32 [B]; dims from :func:`gated_dims`.
    Where y is allocated here, its rows past a sequence's length hold unspecified values."""
    return _gated_forward(x, r, g, lam, dims, B, L, h0, lengths, None, y, h_last, status, stream, check, False)[:2]


def gated_step(x: torch.Tensor, r: torch.Tensor, g: torch.Tensor, lam: torch.Tensor, dims: Dims, state: torch.Tensor,
               new_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, stream=None, check: bool = True) -> torch.Tensor:
    """One position of each of B sequences (x, r, g, y: [B, E]) on their states (fp32 [B, E]), which are updated in
    place unless new_state is given: r2l_gated_scan with L = 1.  A sequence with lengths[b] = 0 keeps its state.
    Returns y."""
    return _gated_forward(x, r, g, lam, dims, state.shape[0], 1, state, lengths, None, y,
                          state if new_state is None else new_state, None, stream, check, False)[0]


def gated_scan_checkpoint_size(dims: Dims, B: int, L: int) -> int:
    return int(load().r2l_gated_scan_checkpoint_size(ctypes.byref(dims), _int(B), _int(L)))


def gated_scan_train(x: torch.Tensor, r: torch.Tensor, g: torch.Tensor, lam: torch.Tensor, dims: Dims, B: int, L: int,
                     h0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                     checkpoint: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                     h_last: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None,
                     check: bool = True):
    """r2l_gated_scan_train: returns (y, h_last, checkpoint); the checkpoint goes to :func:`gated_scan_backward`.
    With R2L_FLAG_ACT8 in dims it also holds x, r and g in 8 bits, which the gradient then reads instead of them."""
    return _gated_forward(x, r, g, lam, dims, B, L, h0, lengths, checkpoint, y, h_last, status, stream, check, True)


def gated_scan_backward_workspace_size(dims: Dims, B: int, L: int) -> int:
    return int(load().r2l_gated_scan_backward_workspace_size(ctypes.byref(dims), _int(B), _int(L)))


def gated_scan_backward(dy: torch.Tensor, lam: torch.Tensor, dims: Dims, B: int, L: int, checkpoint: torch.Tensor,
                        x: Optional[torch.Tensor] = None, r: Optional[torch.Tensor] = None,
                        g: Optional[torch.Tensor] = None, dh_last: Optional[torch.Tensor] = None,
                        lengths: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                        dr: Optional[torch.Tensor] = None, dg: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None,
                        check: bool = True) -> Dict[str, torch.Tensor]:
    """r2l_gated_scan_backward: returns {"dx", "dr", "dg", "dlam", "dh0"} (dx, dr, dg in dims' dtype, [B·L, E],
    allocated here unless given; dlam fp32 [E], dh0 fp32 [B, E]).  x, r and g as given to the forward; with
    R2L_FLAG_ACT8 in dims they are not read and may be left out."""
    lib = load()
    if not dy.is_cuda:
        raise ValueError("libr2l takes device tensors")
    M, E, dtype, dev = _positions(B, L), dims.d_inner, _DTYPES[dims.dtype], dy.device
    if dims.flags & R2L_FLAG_ACT8:
        gi = GatedIn(None, None, None, 0, 0, 0, _vec(lam, (E,), dev, "lam"), None)
    else:
        if x is None or r is None or g is None:
            raise ValueError("x, r and g are needed unless the checkpoint holds them (R2L_FLAG_ACT8)")
        gi = _gated_inputs(x, r, g, lam, None, dims, B, L)
    out = {"dx": dx, "dr": dr, "dg": dg}

    def call(st):
        ws = workspace
        if ws is None:
            ws = torch.empty(gated_scan_backward_workspace_size(dims, B, L), dtype=torch.uint8, device=dev)
        if dx is None and dr is None and dg is None:
            out.update(zip(("dx", "dr", "dg"), torch.empty((3, M, E), dtype=dtype, device=dev).unbind(0)))
        for n, t in out.items():
            if t is None:
                out[n] = torch.empty((M, E), dtype=dtype, device=dev)
        out["dlam"] = torch.empty(E, dtype=torch.float32, device=dev)
        out["dh0"] = torch.empty((B, E), dtype=torch.float32, device=dev)
        (pdx, ldx), (pdr, ldr), (pdg, ldg) = (_rows(out[n], M, E, dtype, dev, n) for n in ("dx", "dr", "dg"))
        gr = GatedGrads(pdx, pdr, pdg, ldx, ldr, ldg, out["dlam"].data_ptr(), out["dh0"].data_ptr())
        pdy, ld_dy = _rows(dy, M, E, dtype, dev, "dy")
        return lib.r2l_gated_scan_backward(gi, pdy, ld_dy, _vec(dh_last, (B, E), dev, "dh_last"), gr, dims, B, L,
                                           _vec(lengths, (B,), dev, "lengths", torch.int32),
                                           *_bytes(checkpoint, dev, "checkpoint"), *_bytes(ws, dev, "workspace"), st)

    rc = _call_on(dev, stream, call)
    if check and rc != 0:
        raise R2LError(rc, "r2l_gated_scan_backward")
    return out


# ---------------------------------------------------------------- 8-bit activation checkpoints

def act8_pack(x: torch.Tensor, B: int, L: int, lengths: Optional[torch.Tensor] = None,
              q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None,
              check: bool = True):
    """r2l_act8_pack of x [B·L, cols] (bf16 or fp32; columns of a wider tensor will do): returns (q, scales), q
    [B·L, cols] torch.float8_e4m3fn and scales [B·L, ⌈cols/64⌉] uint8.  Rows past a sequence's length are not written."""
    lib = load()
    if not x.is_cuda:
        raise ValueError("libr2l takes device tensors")
    if x.dim() != 2 or x.dtype not in _CODES:
        raise ValueError("x must be [B·L, cols], bf16 or fp32")
    M, cols, dev = _positions(B, L), x.shape[1], x.device
    groups = -(-cols // ACT8_GROUP)
    px, ldx = _rows(x, M, cols, x.dtype, dev, "x")

    def call(st):
        nonlocal q, scales
        if q is None:
            q = torch.empty((M, cols), dtype=torch.float8_e4m3fn, device=dev)
        if scales is None:
            scales = torch.empty((M, groups), dtype=torch.uint8, device=dev)
        pq, ldq = _rows(q, M, cols, torch.float8_e4m3fn, dev, "q")
        return lib.r2l_act8_pack(px, ldx, _CODES[x.dtype], B, L, cols, _vec(lengths, (B,), dev, "lengths", torch.int32),
                                 pq, ldq, _vec(scales, (M, groups), dev, "scales", torch.uint8), st)

    rc = _call_on(dev, stream, call)
    if check and rc != 0:
        raise R2LError(rc, "r2l_act8_pack")
    return q, scales


def act8_unpack(q: torch.Tensor, scales: torch.Tensor, B: int, L: int, dtype: torch.dtype = torch.bfloat16,
                lengths: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None,
                check: bool = True) -> torch.Tensor:
    """r2l_act8_unpack: the values that q and scales (from :func:`act8_pack`) stand for, [B·L, cols] in dtype (or in
    out's).  Rows past a sequence's length are not written."""
    lib = load()
    if not q.is_cuda:
        raise ValueError("libr2l takes device tensors")
    if q.dim() != 2:
        raise ValueError("q must be [B·L, cols]")
    M, cols, dev = _positions(B, L), q.shape[1], q.device
    if out is not None:
        dtype = out.dtype
    if dtype not in _CODES:
        raise ValueError("the output is bf16 or fp32")
    pq, ldq = _rows(q, M, cols, torch.float8_e4m3fn, dev, "q")

    def call(st):
        nonlocal out
        if out is None:
            out = torch.empty((M, cols), dtype=dtype, device=dev)
        po, ldo = _rows(out, M, cols, dtype, dev, "out")
        return lib.r2l_act8_unpack(pq, ldq, _vec(scales, (M, -(-cols // ACT8_GROUP)), dev, "scales", torch.uint8),
                                   _CODES[dtype], B, L, cols, _vec(lengths, (B,), dev, "lengths", torch.int32), po, ldo,
                                   st)

    rc = _call_on(dev, stream, call)
    if check and rc != 0:
        raise R2LError(rc, "r2l_act8_unpack")
    return out

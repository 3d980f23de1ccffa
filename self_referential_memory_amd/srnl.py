"""Thin ctypes binding over libsrnl.so (C ABI in include/srnl.h).

Argument marshalling only: tensors are passed as device pointers with the
caller's current HIP stream; every step of the operator runs in the library's
kernels. The library must be built (``python -m
self_referential_memory_amd.build`` or ``__graft_entry__.build()``); loading
fails loudly when it is missing. There is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch
from torch.autograd import forward_ad

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsrnl.so")

SRNL_OK, SRNL_ERR_ARG, SRNL_ERR_DTYPE, SRNL_ERR_PTR, SRNL_ERR_WORKSPACE, SRNL_ERR_HIP = (
    0, -1, -2, -3, -4, -5)
SRNL_ERR_NONFINITE = -6
SRNL_F32, SRNL_BF16 = 0, 1
FLAG_HARD_CAP, FLAG_NO_CAP, FLAG_NO_CLAMP, FLAG_FIXED_ALPHA, FLAG_READ_BEFORE = (
    0x1, 0x2, 0x4, 0x8, 0x10)
FLAG_FREEZE_KV = 0x20
FLAG_CHECK_FINITE = 0x40
FLAG_RECORD = 0x80
ACT_NONE, ACT_GELU, ACT_SILU = 0, 1, 2
ACTS = {"none": ACT_NONE, "gelu": ACT_GELU, "silu": ACT_SILU}

EXPORTS = ("srnl_scan_fwd", "srnl_scan_workspace_bytes", "srnl_scan_1d",
           "srnl_scan_1d_workspace_bytes", "srnl_fuse", "srnl_scan_bwd",
           "srnl_scan_bwd_workspace_bytes", "srnl_scan_1d_bwd", "srnl_scan_1d_bwd_workspace_bytes",
           "srnl_fuse_bwd", "srnl_fuse_bwd_workspace_bytes", "srnl_fuse_bwd_noalloc",
           "srnl_scan_fuse_bwd", "srnl_scan_fuse_bwd_workspace_bytes",
           "srnl_route_gather", "srnl_init_states", "srnl_block_fwd",
           "srnl_block_workspace_bytes",
           "srnl_layer_norm_fwd", "srnl_layer_norm_bwd", "srnl_layer_norm_bwd_workspace_bytes",
           "srnl_linear_fwd", "srnl_linear_bwd", "srnl_linear_bwd_workspace_bytes",
           "srnl_dwconv_fwd", "srnl_dwconv_bwd", "srnl_dwconv_bwd_workspace_bytes",
           "srnl_group_norm_fwd", "srnl_group_norm_fwd_workspace_bytes", "srnl_group_norm_bwd",
           "srnl_group_norm_bwd_workspace_bytes", "srnl_dropout_fwd", "srnl_dropout_bwd",
           "srnl_gated_delta_step", "srnl_gated_delta_fwd", "srnl_gated_delta_fwd_workspace_bytes",
           "srnl_gated_delta_record_bytes", "srnl_gated_delta_bwd",
           "srnl_gated_delta_bwd_workspace_bytes",
           "srnl_route_index", "srnl_chunk_len", "srnl_status_string",
           "srnl_last_error")


class SrnlError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status}: {detail}")
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [("states", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("in_dtype", ctypes.c_int), ("alpha_max", ctypes.c_float),
                ("eps", ctypes.c_float), ("chunk_row", ctypes.c_int),
                ("chunk_col", ctypes.c_int), ("flags", ctypes.c_uint),
                ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class BlockWeights(ctypes.Structure):
    """srnl_block_weights: device pointers of the block parameters."""
    _fields_ = [("ln1_w", ctypes.c_void_p), ("ln1_b", ctypes.c_void_p),
                ("wq", ctypes.c_void_p), ("dw_w", ctypes.c_void_p), ("dw_b", ctypes.c_void_p),
                ("ln2_w", ctypes.c_void_p), ("ln2_b", ctypes.c_void_p),
                ("w1", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("b2", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("ffn_hidden", ctypes.c_int),
                ("ln_eps", ctypes.c_float)]


class LinearParams(ctypes.Structure):
    """srnl_linear_params."""
    _fields_ = [("w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("x_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
                ("residual_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("stream", ctypes.c_void_p)]


class GatedDeltaParams(ctypes.Structure):
    """srnl_gated_delta_params."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "g", "beta", "state", "lengths")]
                + [(n, ctypes.c_int) for n in ("B", "T", "Hk", "H", "Dk", "Dv")]
                + [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "v_stride")]
                + [("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("norm_eps", ctypes.c_float),
                   ("stream", ctypes.c_void_p)])


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsrnl.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, u = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint
        L.srnl_scan_fwd.argtypes = [vp, i, i, i, i, i, i, u, ctypes.POINTER(Params), vp]
        L.srnl_scan_1d.argtypes = [vp, i, i, i, i, i, ctypes.POINTER(Params), vp]
        L.srnl_fuse.argtypes = [vp, i, i, i, i, u, vp, i, vp, vp]
        sz = ctypes.c_size_t
        L.srnl_scan_workspace_bytes.argtypes = [i, i, i, i, i, i, u, ctypes.POINTER(Params)]
        L.srnl_scan_workspace_bytes.restype = sz
        L.srnl_scan_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, u, ctypes.POINTER(Params)]
        L.srnl_scan_bwd_workspace_bytes.restype = sz
        L.srnl_scan_bwd.argtypes = [vp, i, i, i, i, i, i, u, ctypes.POINTER(Params), vp, vp, sz,
                                    vp, vp, vp]
        L.srnl_scan_1d_workspace_bytes.argtypes = [i, i, i, i, i, ctypes.POINTER(Params)]
        L.srnl_scan_1d_workspace_bytes.restype = sz
        L.srnl_scan_1d_bwd_workspace_bytes.argtypes = [i, i, i, i, i, ctypes.POINTER(Params)]
        L.srnl_scan_1d_bwd_workspace_bytes.restype = sz
        L.srnl_scan_1d_bwd.argtypes = [vp, i, i, i, i, i, ctypes.POINTER(Params), vp, vp, sz,
                                       vp, vp, vp]
        L.srnl_fuse_bwd_workspace_bytes.argtypes = [i, i, i, i, u]
        L.srnl_fuse_bwd_workspace_bytes.restype = sz
        L.srnl_fuse_bwd.argtypes = [vp, vp, i, i, i, i, u, vp, vp, vp, vp, sz, vp]
        L.srnl_fuse_bwd_noalloc.argtypes = [vp, vp, i, i, i, i, u, vp, vp, vp, vp]
        L.srnl_scan_fuse_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, u, ctypes.POINTER(Params)]
        L.srnl_scan_fuse_bwd_workspace_bytes.restype = sz
        L.srnl_scan_fuse_bwd.argtypes = [vp, i, i, i, i, i, i, u, ctypes.POINTER(Params), vp, vp,
                                         vp, vp, sz, vp, vp, vp, vp]
        L.srnl_route_gather.argtypes = [vp, i, i, i, i, u, i, vp, vp]
        L.srnl_init_states.argtypes = [vp, i, i, ctypes.c_ulonglong, ctypes.c_float, vp]
        L.srnl_block_workspace_bytes.argtypes = [i, i, i, i, u]
        L.srnl_block_workspace_bytes.restype = sz
        L.srnl_block_fwd.argtypes = [vp, i, i, i, i, i, i, u, ctypes.POINTER(Params),
                                     ctypes.POINTER(BlockWeights), vp, sz, vp]
        ll, lp = ctypes.c_longlong, ctypes.POINTER(LinearParams)
        L.srnl_layer_norm_fwd.argtypes = [vp, ll, i, i, vp, vp, ctypes.c_float, i, vp, vp, vp, vp]
        L.srnl_layer_norm_bwd.argtypes = [vp, i, vp, ll, i, i, vp, vp, vp, vp, i, vp, vp, vp, vp,
                                          sz, vp]
        L.srnl_layer_norm_bwd_workspace_bytes.argtypes = [ll, i]
        L.srnl_layer_norm_bwd_workspace_bytes.restype = sz
        L.srnl_linear_fwd.argtypes = [vp, ll, i, i, lp, vp, vp]
        L.srnl_linear_bwd.argtypes = [vp, vp, ll, i, i, lp, vp, vp, vp, vp, vp, vp, sz]
        L.srnl_linear_bwd_workspace_bytes.argtypes = [ll, i, i, lp]
        L.srnl_linear_bwd_workspace_bytes.restype = sz
        L.srnl_dwconv_fwd.argtypes = [vp, i, i, i, i, i, vp, vp, vp, i, vp, i, i, vp, vp]
        L.srnl_dwconv_bwd.argtypes = [vp, i, vp, i, i, i, i, i, vp, vp, vp, vp, vp, vp, sz, vp]
        L.srnl_dwconv_bwd_workspace_bytes.argtypes = [i, i, i, i]
        L.srnl_dwconv_bwd_workspace_bytes.restype = sz
        L.srnl_group_norm_fwd_workspace_bytes.argtypes = [i, ll, i, i]
        L.srnl_group_norm_fwd_workspace_bytes.restype = sz
        L.srnl_group_norm_fwd.argtypes = [vp, i, ll, i, i, i, vp, vp, ctypes.c_float, i, i, vp, vp,
                                          vp, vp, sz, vp]
        L.srnl_group_norm_bwd_workspace_bytes.argtypes = [i, ll, i, i]
        L.srnl_group_norm_bwd_workspace_bytes.restype = sz
        L.srnl_group_norm_bwd.argtypes = [vp, i, vp, i, ll, i, i, i, vp, vp, vp, vp, i, vp, vp, vp,
                                          vp, vp, sz, vp]
        ull = ctypes.c_ulonglong
        L.srnl_dropout_fwd.argtypes = [vp, i, ll, ctypes.c_double, ull, ull, vp, vp, i, i, vp, vp]
        L.srnl_dropout_bwd.argtypes = [vp, i, ll, ctypes.c_double, ull, ull, vp, vp, i, vp, vp]
        dp = ctypes.POINTER(GatedDeltaParams)
        L.srnl_gated_delta_step.argtypes = [dp, vp, vp]
        L.srnl_gated_delta_fwd.argtypes = [dp, vp, vp, vp, sz, vp, sz]
        L.srnl_gated_delta_bwd.argtypes = [dp, vp, vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, sz]
        for f in ("srnl_gated_delta_record_bytes", "srnl_gated_delta_fwd_workspace_bytes",
                  "srnl_gated_delta_bwd_workspace_bytes"):
            getattr(L, f).argtypes = [dp]
            getattr(L, f).restype = sz
        for f in ("srnl_layer_norm_fwd", "srnl_layer_norm_bwd", "srnl_linear_fwd",
                  "srnl_linear_bwd", "srnl_dwconv_fwd", "srnl_dwconv_bwd", "srnl_group_norm_fwd",
                  "srnl_group_norm_bwd", "srnl_dropout_fwd", "srnl_dropout_bwd",
                  "srnl_gated_delta_step", "srnl_gated_delta_fwd", "srnl_gated_delta_bwd"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("srnl_scan_fwd", "srnl_scan_1d", "srnl_fuse", "srnl_scan_bwd",
                  "srnl_scan_1d_bwd", "srnl_fuse_bwd", "srnl_fuse_bwd_noalloc",
                  "srnl_scan_fuse_bwd", "srnl_route_gather", "srnl_init_states", "srnl_block_fwd"):
            getattr(L, f).restype = ctypes.c_int
        L.srnl_route_index.argtypes = [i, i, i, ctypes.c_long, ctypes.POINTER(i),
                                       ctypes.POINTER(i)]
        L.srnl_route_index.restype = None
        L.srnl_chunk_len.argtypes = [i, i, i, i, i]
        L.srnl_chunk_len.restype = ctypes.c_int
        L.srnl_status_string.argtypes = [i]
        L.srnl_status_string.restype = ctypes.c_char_p
        L.srnl_last_error.argtypes = []
        L.srnl_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != SRNL_OK:
        raise SrnlError(status, where, lib().srnl_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _expect(t: Optional[torch.Tensor], shape, dtype, name: str) -> None:
    """The library sees only pointers: buffer shapes and dtypes are checked here."""
    if t is None:
        return
    if t.shape != (shape if isinstance(shape, tuple) else tuple(shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _state_shape(heads: int, d: int):
    return (4, heads, 3 * d * d + 2 * d)


def _stream(stream, x: Optional[torch.Tensor] = None) -> int:
    """The handle of stream (None: the current device's current one), which
    must be of x's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if x is not None and stream.device_index != x.get_device():
        raise ValueError(f"stream of cuda:{stream.device_index}, tensors on {x.device}")
    return stream.cuda_stream


def _keep_for_stream(handle, *tensors) -> None:
    """Temporaries this binding allocates (on the current stream) and frees
    on return, but whose kernels run on the stream ``handle``: record that
    stream on them, so the caching allocator does not hand their memory out
    again before that stream's work is done."""
    if (handle or 0) == (_stream(None) or 0):
        return
    s = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    for t in tensors:
        if t is not None:
            t.record_stream(s)


_DTYPE_CODES = {torch.float32: SRNL_F32, torch.bfloat16: SRNL_BF16}


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return code


def route_index(r: int, H: int, W: int, t: int):
    i, j = ctypes.c_int(), ctypes.c_int()
    lib().srnl_route_index(r, H, W, t, ctypes.byref(i), ctypes.byref(j))
    return i.value, j.value


def chunk_len(r: int, H: int, W: int, chunk_row: int = 0, chunk_col: int = 0) -> int:
    return lib().srnl_chunk_len(r, H, W, chunk_row, chunk_col)


def make_params(states: torch.Tensor, x: torch.Tensor, q: Optional[torch.Tensor] = None, *,
                alpha_max: float = 0.9, eps: float = 1e-6, chunk_row: int = 0,
                chunk_col: int = 0, flags: int = 0, stream=None) -> Params:
    if q is not None and (q.dtype != x.dtype or q.shape != x.shape):
        raise SrnlError(SRNL_ERR_DTYPE, "make_params",
                        "separate queries must have the shape and dtype of x")
    return Params(_ptr(states), _ptr(q), _dtype_code(x), alpha_max, eps, chunk_row,
                  chunk_col, flags, _stream(stream))


def _finite_check_workspace(p: Params, x: torch.Tensor, nbytes: int):
    """With SRNL_FLAG_CHECK_FINITE and no caller workspace, allocate one of
    nbytes (the entry point's workspace query) and point p at it; the call
    waits for its stream when checking, so the buffer outlives its use.
    Returns the tensor (None when nothing was allocated). A record
    (SRNL_FLAG_RECORD) must outlive the call: that takes scan_fwd_record
    (scan_1d_record) or a caller workspace."""
    if p.workspace or not nbytes:
        return None
    if p.flags & FLAG_RECORD and nbytes > (256 if p.flags & FLAG_CHECK_FINITE else 0):
        raise ValueError("FLAG_RECORD needs a workspace that outlives the call: use "
                         "scan_fwd_record (scan_1d_record), which returns the record, or "
                         "pass params with a workspace")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    p.workspace, p.workspace_bytes = ws.data_ptr(), nbytes
    return ws


def scan_fwd(x: torch.Tensor, states: torch.Tensor, heads: int, d: int,
             route_mask: int = 15, q: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, *, params: Optional[Params] = None,
             **kw) -> torch.Tensor:
    """srnl_scan_fwd: x [B,H,W,C] -> per-route outputs [R,B,H*W,C] fp32."""
    B, H, W, C = x.shape
    R = bin(route_mask & 15).count("1")
    _expect(states, _state_shape(heads, d), torch.float32, "states")
    if out is None:
        out = torch.empty((R, B, H * W, C), dtype=torch.float32, device=x.device)
    _expect(out, (R, B, H * W, C), torch.float32, "out")
    p = params if params is not None else make_params(states, x, q, **kw)
    nbytes = 0 if p.workspace else lib().srnl_scan_workspace_bytes(
        B, H, W, C, heads, d, route_mask, ctypes.byref(p))
    ws = _finite_check_workspace(p, x, nbytes)
    try:
        _check(lib().srnl_scan_fwd(_ptr(x), B, H, W, C, heads, d, route_mask,
                                   ctypes.byref(p), _ptr(out)), "srnl_scan_fwd")
    finally:
        if ws is not None:
            p.workspace, p.workspace_bytes = None, 0
    return out


def scan_fwd_record(x: torch.Tensor, states: torch.Tensor, heads: int, d: int,
                    route_mask: int = 15, q: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, *, flags: int = 0, **kw):
    """srnl_scan_fwd with SRNL_FLAG_RECORD: the route outputs [R,B,H*W,C] and
    the forward record (a uint8 device tensor, or None where the windowed
    backward does not apply) for scan_bwd(..., record=...)."""
    B, H, W, C = x.shape
    R = bin(route_mask & 15).count("1")
    _expect(states, _state_shape(heads, d), torch.float32, "states")
    if out is None:
        out = torch.empty((R, B, H * W, C), dtype=torch.float32, device=x.device)
    _expect(out, (R, B, H * W, C), torch.float32, "out")
    p = make_params(states, x, q, flags=flags | FLAG_RECORD, **kw)
    only = Params.from_buffer_copy(p)
    only.flags &= ~FLAG_CHECK_FINITE
    rec_bytes = lib().srnl_scan_workspace_bytes(B, H, W, C, heads, d, route_mask,
                                                ctypes.byref(only))
    nbytes = lib().srnl_scan_workspace_bytes(B, H, W, C, heads, d, route_mask, ctypes.byref(p))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    if ws is not None:
        p.workspace, p.workspace_bytes = ws.data_ptr(), nbytes
    _check(lib().srnl_scan_fwd(_ptr(x), B, H, W, C, heads, d, route_mask, ctypes.byref(p),
                               _ptr(out)), "srnl_scan_fwd")
    rec = ws[:rec_bytes] if rec_bytes else None
    return out, rec


def scan_1d(x: torch.Tensor, states: torch.Tensor, heads: int, d: int,
            q: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, *,
            chunk: int = 0, params: Optional[Params] = None, **kw) -> torch.Tensor:
    """srnl_scan_1d: x [B,N,C] -> y [B,N,C] fp32 (chunk 0 selects 64 tokens)."""
    B, N, C = x.shape
    _expect(states, (heads, 3 * d * d + 2 * d), torch.float32, "states")
    if out is None:
        out = torch.empty((B, N, C), dtype=torch.float32, device=x.device)
    _expect(out, (B, N, C), torch.float32, "out")
    p = params if params is not None else make_params(states, x, q, chunk_row=chunk, **kw)
    nbytes = 0 if p.workspace else lib().srnl_scan_1d_workspace_bytes(
        B, N, C, heads, d, ctypes.byref(p))
    ws = _finite_check_workspace(p, x, nbytes)
    try:
        _check(lib().srnl_scan_1d(_ptr(x), B, N, C, heads, d, ctypes.byref(p), _ptr(out)),
               "srnl_scan_1d")
    finally:
        if ws is not None:
            p.workspace, p.workspace_bytes = None, 0
    return out


def scan_1d_record(x: torch.Tensor, states: torch.Tensor, heads: int, d: int,
                   q: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, *,
                   chunk: int = 0, flags: int = 0, **kw):
    """srnl_scan_1d with SRNL_FLAG_RECORD: y [B,N,C] and the forward record
    (a uint8 device tensor, or None where the windowed backward does not
    apply) for scan_1d_bwd(..., record=...)."""
    B, N, C = x.shape
    _expect(states, (heads, 3 * d * d + 2 * d), torch.float32, "states")
    if out is None:
        out = torch.empty((B, N, C), dtype=torch.float32, device=x.device)
    _expect(out, (B, N, C), torch.float32, "out")
    p = make_params(states, x, q, chunk_row=chunk, flags=flags | FLAG_RECORD, **kw)
    only = Params.from_buffer_copy(p)
    only.flags &= ~FLAG_CHECK_FINITE
    rec_bytes = lib().srnl_scan_1d_workspace_bytes(B, N, C, heads, d, ctypes.byref(only))
    nbytes = lib().srnl_scan_1d_workspace_bytes(B, N, C, heads, d, ctypes.byref(p))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    if ws is not None:
        p.workspace, p.workspace_bytes = ws.data_ptr(), nbytes
    _check(lib().srnl_scan_1d(_ptr(x), B, N, C, heads, d, ctypes.byref(p), _ptr(out)),
           "srnl_scan_1d")
    return out, (ws[:rec_bytes] if rec_bytes else None)


def scan_1d_bwd(x: torch.Tensor, states: torch.Tensor, heads: int, d: int, dy: torch.Tensor,
                q: Optional[torch.Tensor] = None, *, chunk: int = 0,
                record: Optional[torch.Tensor] = None, **kw):
    """srnl_scan_1d_bwd: dy [B,N,C] fp32 -> (dx [B,N,C], dq or None, dstates
    [heads,3d^2+2d]), all fp32, for srnl_scan_1d's forward with the same
    arguments (chunk 0 selects 64 tokens). ``record``: the forward record
    from scan_1d_record. The workspace is allocated here (torch)."""
    B, N, C = x.shape
    _expect(states, (heads, 3 * d * d + 2 * d), torch.float32, "states")
    _expect(dy, (B, N, C), torch.float32, "dy")
    p = make_params(states, x, q, chunk_row=chunk, **kw)
    if record is not None:
        p.flags = (p.flags | FLAG_RECORD) & ~FLAG_CHECK_FINITE
        p.workspace, p.workspace_bytes = record.data_ptr(), record.numel() * record.element_size()
    nbytes = lib().srnl_scan_1d_bwd_workspace_bytes(B, N, C, heads, d, ctypes.byref(p))
    ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=x.device)
    dx = torch.empty((B, N, C), dtype=torch.float32, device=x.device)
    dq = None if q is None else torch.empty_like(dx)
    dst = torch.empty((heads, 3 * d * d + 2 * d), dtype=torch.float32, device=x.device)
    _check(lib().srnl_scan_1d_bwd(_ptr(x), B, N, C, heads, d, ctypes.byref(p), _ptr(dy),
                                  _ptr(ws), int(nbytes), _ptr(dx), _ptr(dq), _ptr(dst)),
           "srnl_scan_1d_bwd")
    _keep_for_stream(p.stream, ws)
    return dx, dq, dst


def fuse(y: torch.Tensor, B: int, H: int, W: int, C: int, route_mask: int,
         scales: torch.Tensor, out_dtype=torch.float32, out: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """srnl_fuse: per-route outputs -> restored, channel-scaled sum [B,H,W,C]."""
    R = bin(route_mask & 15).count("1")
    _expect(y, (R, B, H * W, C), torch.float32, "y")
    _expect(scales, (4, C), torch.float32, "scales")
    if out is None:
        out = torch.empty((B, H, W, C), dtype=out_dtype, device=y.device)
    _check(lib().srnl_fuse(_ptr(y), B, H, W, C, route_mask, _ptr(scales),
                           _dtype_code(out), _ptr(out), _stream(stream)), "srnl_fuse")
    return out


def scan_bwd(x: torch.Tensor, states: torch.Tensor, heads: int, d: int, dy: torch.Tensor,
             route_mask: int = 15, q: Optional[torch.Tensor] = None, *,
             params: Optional[Params] = None, record: Optional[torch.Tensor] = None, **kw):
    """srnl_scan_bwd: dy [R,B,H*W,C] fp32 -> (dx [B,H,W,C], dq or None, dstates
    [4,heads,3d^2+2d]), all fp32. The workspace is allocated here (torch).
    ``record``: the forward record from scan_fwd_record with the same
    arguments; the backward then reads it instead of recomputing it."""
    B, H, W, C = x.shape
    R = bin(route_mask & 15).count("1")
    _expect(states, _state_shape(heads, d), torch.float32, "states")
    _expect(dy, (R, B, H * W, C), torch.float32, "dy")
    p = params if params is not None else make_params(states, x, q, **kw)
    if record is not None:
        p = Params.from_buffer_copy(p)
        p.flags = (p.flags | FLAG_RECORD) & ~FLAG_CHECK_FINITE
        p.workspace, p.workspace_bytes = record.data_ptr(), record.numel() * record.element_size()
    nbytes = lib().srnl_scan_bwd_workspace_bytes(B, H, W, C, heads, d, route_mask, ctypes.byref(p))
    ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=x.device)
    dx = torch.empty((B, H, W, C), dtype=torch.float32, device=x.device)
    dq = None if q is None else torch.empty_like(dx)
    dst = torch.empty((4, heads, 3 * d * d + 2 * d), dtype=torch.float32, device=x.device)
    _check(lib().srnl_scan_bwd(_ptr(x), B, H, W, C, heads, d, route_mask, ctypes.byref(p),
                               _ptr(dy), _ptr(ws), int(nbytes), _ptr(dx), _ptr(dq), _ptr(dst)),
           "srnl_scan_bwd")
    _keep_for_stream(p.stream, ws)
    return dx, dq, dst


def fuse_bwd(dout: torch.Tensor, y: torch.Tensor, B: int, H: int, W: int, C: int,
             route_mask: int, scales: torch.Tensor, stream=None):
    """srnl_fuse_bwd: dout [B,H,W,C] fp32 -> (dy_routes [R,B,H*W,C], dscales [4,C])."""
    R = bin(route_mask & 15).count("1")
    _expect(dout, (B, H, W, C), torch.float32, "dout")
    _expect(y, (R, B, H * W, C), torch.float32, "y")
    _expect(scales, (4, C), torch.float32, "scales")
    nbytes = lib().srnl_fuse_bwd_workspace_bytes(B, H, W, C, route_mask)
    ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=dout.device)
    dyr = torch.empty_like(y)
    dsc = torch.empty((4, C), dtype=torch.float32, device=dout.device)
    sh = _stream(stream)
    _check(lib().srnl_fuse_bwd(_ptr(dout), _ptr(y), B, H, W, C, route_mask, _ptr(scales),
                               _ptr(dyr), _ptr(dsc), _ptr(ws), int(nbytes), sh),
           "srnl_fuse_bwd")
    _keep_for_stream(sh, ws)
    return dyr, dsc


def scan_fuse_bwd(x: torch.Tensor, states: torch.Tensor, heads: int, d: int, y: torch.Tensor,
                  scales: torch.Tensor, dout: torch.Tensor, route_mask: int = 15,
                  q: Optional[torch.Tensor] = None, *, params: Optional[Params] = None,
                  record: Optional[torch.Tensor] = None, **kw):
    """srnl_scan_fuse_bwd: the operator's backward in one call, dout [B,H,W,C]
    fp32 -> (dx [B,H,W,C], dq or None, dstates [4,heads,3d^2+2d], dscales
    [4,C]), all fp32; the same results as fuse_bwd then scan_bwd. y: the
    forward's route outputs [R,B,H*W,C]; ``record`` as for scan_bwd."""
    B, H, W, C = x.shape
    R = bin(route_mask & 15).count("1")
    _expect(states, _state_shape(heads, d), torch.float32, "states")
    _expect(y, (R, B, H * W, C), torch.float32, "y")
    _expect(scales, (4, C), torch.float32, "scales")
    _expect(dout, (B, H, W, C), torch.float32, "dout")
    p = params if params is not None else make_params(states, x, q, **kw)
    if record is not None:
        p = Params.from_buffer_copy(p)
        p.flags = (p.flags | FLAG_RECORD) & ~FLAG_CHECK_FINITE
        p.workspace, p.workspace_bytes = record.data_ptr(), record.numel() * record.element_size()
    nbytes = lib().srnl_scan_fuse_bwd_workspace_bytes(B, H, W, C, heads, d, route_mask,
                                                      ctypes.byref(p))
    ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=x.device)
    dx = torch.empty((B, H, W, C), dtype=torch.float32, device=x.device)
    dq = None if q is None else torch.empty_like(dx)
    dst = torch.empty((4, heads, 3 * d * d + 2 * d), dtype=torch.float32, device=x.device)
    dsc = torch.empty((4, C), dtype=torch.float32, device=x.device)
    _check(lib().srnl_scan_fuse_bwd(_ptr(x), B, H, W, C, heads, d, route_mask, ctypes.byref(p),
                                    _ptr(y), _ptr(scales), _ptr(dout), _ptr(ws), int(nbytes),
                                    _ptr(dx), _ptr(dq), _ptr(dst), _ptr(dsc)),
           "srnl_scan_fuse_bwd")
    _keep_for_stream(p.stream, ws)
    return dx, dq, dst, dsc


def route_gather(x: torch.Tensor, route_mask: int = 15, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """srnl_route_gather: x [B,H,W,C] -> [R,B,H*W,C] in route order."""
    B, H, W, C = x.shape
    R = bin(route_mask & 15).count("1")
    if out is None:
        out = torch.empty((R, B, H * W, C), dtype=x.dtype, device=x.device)
    _check(lib().srnl_route_gather(_ptr(x), B, H, W, C, route_mask, _dtype_code(x),
                                   _ptr(out), _stream(stream)), "srnl_route_gather")
    return out


def init_states(heads: int, d: int, seed: int, std: float, device="cuda",
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """srnl_init_states: [4, heads, 3d^2+2d] fp32 ~ std * N(0,1) (Philox)."""
    if out is None:
        out = torch.empty((4, heads, 3 * d * d + 2 * d), dtype=torch.float32, device=device)
    _check(lib().srnl_init_states(_ptr(out), heads, d, seed, std, _stream(stream)),
           "srnl_init_states")
    return out


def forward(x: torch.Tensor, states: torch.Tensor, scales: torch.Tensor, heads: int, d: int,
            route_mask: int = 15, q: Optional[torch.Tensor] = None, out_dtype=None,
            **kw) -> torch.Tensor:
    """Scan + fuse: the operator's forward pass on an NHWC grid."""
    B, H, W, C = x.shape
    y = scan_fwd(x, states, heads, d, route_mask, q, **kw)
    return fuse(y, B, H, W, C, route_mask, scales,
                out_dtype=x.dtype if out_dtype is None else out_dtype,
                stream=kw.get("stream"))


def _side_stream(kw):
    """The stream kw asks for when it is not the current one, else None."""
    s = kw.get("stream")
    if s is None:
        return None
    cur = torch.cuda.current_stream()
    return None if (s.cuda_stream or 0) == (cur.cuda_stream or 0) else s


class Operator(torch.autograd.Function):
    """The operator (scan + fuse) as an autograd node: the forward pass is
    srnl_scan_fwd and srnl_fuse, the backward pass srnl_scan_fuse_bwd (the
    results of srnl_fuse_bwd then srnl_scan_bwd). Gradients flow to x, the initial states, the scales and
    the separate queries. The route outputs are kept for the fusion backward,
    and, where the windowed backward applies, the forward's record
    (SRNL_FLAG_RECORD), so the backward does not run the forward again.

    With stream= (kw) another than the current stream, both passes run on
    that stream: it first waits for the current stream (the inputs, or the
    incoming gradient, are made there), everything the pass allocates is
    allocated on it, and the current stream then waits for it before the
    result is handed back; the results are recorded as used on the current
    stream, so the caching allocator keeps them until that stream is done."""

    @staticmethod
    def forward(ctx, x, states, scales, q, heads, d, route_mask, kw):
        B, H, W, C = x.shape
        side = _side_stream(kw)
        kwc = {k: v for k, v in kw.items() if k != "stream"}
        cur = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(cur)
        with torch.cuda.stream(side if side is not None else cur):
            y, rec = scan_fwd_record(x, states, heads, d, route_mask, q, **kwc)
            out = fuse(y, B, H, W, C, route_mask, scales, out_dtype=x.dtype)
        if side is not None:
            cur.wait_stream(side)
            out.record_stream(cur)
        ctx.save_for_backward(x, states, scales, q, y, rec)
        ctx.cfg = (heads, d, route_mask, kw)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, states, scales, q, y, rec = ctx.saved_tensors
        heads, d, route_mask, kw = ctx.cfg
        B, H, W, C = x.shape
        side = _side_stream(kw)
        kwc = {k: v for k, v in kw.items() if k != "stream"}
        cur = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(cur)
            dout.record_stream(side)
        with torch.cuda.stream(side if side is not None else cur):
            d32 = dout.to(torch.float32).contiguous()
            dx, dq, dst, dsc = scan_fuse_bwd(x, states, heads, d, y, scales, d32, route_mask, q,
                                             record=rec, **kwc)
            grads = (dx.to(x.dtype), dst, dsc, None if dq is None else dq.to(q.dtype))
        if side is not None:
            cur.wait_stream(side)
            for g in grads:
                if g is not None:
                    g.record_stream(cur)
        return grads + (None, None, None, None)


def operator(x: torch.Tensor, states: torch.Tensor, scales: torch.Tensor, heads: int, d: int,
             route_mask: int = 15, q: Optional[torch.Tensor] = None, **kw) -> torch.Tensor:
    """Differentiable scan + fuse on an NHWC grid; the output has x's dtype.
    ``kw`` are the srnl_params fields (alpha_max, eps, chunk_row, chunk_col,
    flags)."""
    return Operator.apply(x, states, scales, q, heads, d, route_mask, kw)


def block_weights(bw: dict, scales: torch.Tensor, ln_eps: float = 1e-5) -> BlockWeights:
    """srnl_block_weights from a dict of device tensors: ln1_w, ln1_b, dw_w
    [C,3,3], dw_b, ln2_w, ln2_b, b1, b2 (fp32) and wq [C,C], w1 [F,C], w2
    [C,F] (bf16). The tensors must outlive the calls that use the struct."""
    # the library sees only pointers: every shape is checked here
    C = int(bw["wq"].shape[0])
    F = int(bw["w1"].shape[0])
    shapes = {"ln1_w": (C,), "ln1_b": (C,), "wq": (C, C), "dw_w": (C, 3, 3), "dw_b": (C,),
              "ln2_w": (C,), "ln2_b": (C,), "w1": (F, C), "b1": (F,), "w2": (C, F), "b2": (C,)}
    for k, shp in shapes.items():
        if tuple(bw[k].shape) != shp:
            raise ValueError(f"{k} has shape {tuple(bw[k].shape)}, expected {shp}")
        want = torch.bfloat16 if k in ("wq", "w1", "w2") else torch.float32
        if bw[k].dtype != want:
            raise ValueError(f"{k} must be {want}")
    if tuple(scales.shape) != (4, C) or scales.dtype != torch.float32:
        raise ValueError(f"scales must be float32 of shape (4, {C})")
    w = BlockWeights(_ptr(bw["ln1_w"]), _ptr(bw["ln1_b"]), _ptr(bw["wq"]), _ptr(bw["dw_w"]),
                     _ptr(bw["dw_b"]), _ptr(bw["ln2_w"]), _ptr(bw["ln2_b"]), _ptr(bw["w1"]),
                     _ptr(bw["b1"]), _ptr(bw["w2"]), _ptr(bw["b2"]), _ptr(scales), F, ln_eps)
    w.channels = C
    return w


def block_fwd(x: torch.Tensor, states: torch.Tensor, weights: BlockWeights, heads: int, d: int,
              route_mask: int = 15, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, *, params: Optional[Params] = None,
              **kw) -> torch.Tensor:
    """srnl_block_fwd: one residual block, x [B,H,W,C] -> out [B,H,W,C] in
    x's dtype. The workspace is allocated here (torch) unless given."""
    B, H, W, C = x.shape
    if getattr(weights, "channels", C) != C:
        raise ValueError(f"weights are for C = {weights.channels}, x has C = {C}")
    _expect(states, _state_shape(heads, d), torch.float32, "states")
    if out is None:
        out = torch.empty_like(x)
    _expect(out, x.shape, x.dtype, "out")
    nbytes = lib().srnl_block_workspace_bytes(B, H, W, C, route_mask)
    if workspace is not None and workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace smaller than srnl_block_workspace_bytes")
    own = workspace is None
    if own:
        workspace = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=x.device)
    p = params if params is not None else make_params(states, x, **kw)
    _check(lib().srnl_block_fwd(_ptr(x), B, H, W, C, heads, d, route_mask, ctypes.byref(p),
                                ctypes.byref(weights), _ptr(workspace),
                                int(workspace.numel() * workspace.element_size()),
                                _ptr(out)), "srnl_block_fwd")
    if own:
        _keep_for_stream(p.stream, workspace)
    return out


# ------------------------------------------------------------ layers

_HERE = contextlib.nullcontext()


def _on(x: torch.Tensor, *others: Optional[torch.Tensor]):
    """The context in which x's device is current (the library launches on the
    current device); every tensor must be on it."""
    i = x.get_device()
    if i < 0:
        raise ValueError("tensors must be on the GPU (there is no CPU path)")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError(f"tensors on {x.device} and {t.device}")
    return _HERE if i == torch._C._cuda_getDevice() else torch.cuda.device(i)


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _new(out: Optional[torch.Tensor], shape, dtype, device, name: str = "out",
         like: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The caller's output, or a new one; like: an input of the same shape
    (contiguous, as _ptr sees to), from which it is made in less host time."""
    if out is None:
        return (torch.empty(shape, dtype=dtype, device=device) if like is None
                else torch.empty_like(like, dtype=dtype))
    _expect(out, shape, dtype, name)
    if out.device != device:
        raise ValueError(f"{name} is on {out.device}, expected {device}")
    return out


def layer_norm_fwd(x: torch.Tensor, gain: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                   eps: float = 1e-5, *, out_dtype=None, stats: bool = False,
                   out: Optional[torch.Tensor] = None, stream=None):
    """srnl_layer_norm_fwd over the last axis of x [..., C] -> y in out_dtype
    (x's when None); with stats also (mean, rstd) [...] fp32, which
    layer_norm_bwd takes. gain, bias: [C] fp32 or None."""
    C = x.shape[-1]
    for t, name in ((gain, "gain"), (bias, "bias")):
        _expect(t, (C,), torch.float32, name)
    dtx = _dtype_code(x)
    with _on(x, gain, bias):
        out = _new(out, x.shape, x.dtype if out_dtype is None else out_dtype, x.device, like=x)
        dto = _dtype_code(out)
        mean = rstd = None
        if stats:
            mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
            rstd = torch.empty_like(mean)
        _check(lib().srnl_layer_norm_fwd(_ptr(x), x.numel() // max(C, 1), C, dtx, _ptr(gain), _ptr(bias),
                                         eps, dto, _ptr(out), _ptr(mean), _ptr(rstd),
                                         _stream(stream, x)), "srnl_layer_norm_fwd")
    return (out, mean, rstd) if stats else out


def layer_norm_bwd(dout: torch.Tensor, x: torch.Tensor, gain: Optional[torch.Tensor],
                   mean: torch.Tensor, rstd: torch.Tensor, *,
                   dx_add: Optional[torch.Tensor] = None, param_grads: bool = True,
                   dx: Optional[torch.Tensor] = None, stream=None):
    """srnl_layer_norm_bwd: dout [..., C] -> (dx in x's dtype, dgain, dbias
    [C] fp32; the last two None without param_grads). dx_add: a gradient of
    x's shape, fp32 or bf16, added to dx (the residual around the norm)."""
    C = x.shape[-1]
    _expect(gain, (C,), torch.float32, "gain")
    _expect(dout, x.shape, None, "dout")
    _expect(dx_add, x.shape, None, "dx_add")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _expect(t, x.shape[:-1], torch.float32, name)
    rows = x.numel() // max(C, 1)
    dtx, dto = _dtype_code(x), _dtype_code(dout)
    dta = 0 if dx_add is None else _dtype_code(dx_add)
    with _on(x, dout, gain, mean, rstd, dx_add):
        dx = _new(dx, x.shape, x.dtype, x.device, "dx", x)
        dgain = dbias = ws = None
        if param_grads:
            dgain = torch.empty(C, dtype=torch.float32, device=x.device)
            dbias = torch.empty_like(dgain)
            ws = _workspace(lib().srnl_layer_norm_bwd_workspace_bytes(rows, C), x.device)
        sh = _stream(stream, x)
        _check(lib().srnl_layer_norm_bwd(
            _ptr(dout), dto, _ptr(x), rows, C, dtx, _ptr(gain), _ptr(mean), _ptr(rstd),
            _ptr(dx_add), dta, _ptr(dx), _ptr(dgain), _ptr(dbias), _ptr(ws),
            0 if ws is None else ws.numel(), sh), "srnl_layer_norm_bwd")
        _keep_for_stream(sh, ws)
    return dx, dgain, dbias


def _act_code(act) -> int:
    if act in ACTS:
        return ACTS[act]
    if isinstance(act, int) and act in ACTS.values():
        return act
    raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")


def linear_fwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               act="none", residual: Optional[torch.Tensor] = None, out_dtype=None,
               keep_pre: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """srnl_linear_fwd: act(x w^T + bias) + residual, x [..., K], w [N, K],
    bias [N] fp32, residual [..., N], each of x, w, residual and the output
    (out_dtype, x's when None) fp32 or bf16. act: "none", "gelu" (erf) or
    "silu". keep_pre: also return x w^T + bias in fp32, which linear_bwd
    takes."""
    N, K = w.shape
    if x.shape[-1] != K:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [..., {K}]")
    shape = x.shape[:-1] + (N,)
    _expect(bias, (N,), torch.float32, "bias")
    _expect(residual, shape, None, "residual")
    code = _act_code(act)
    dtr = 0 if residual is None else _dtype_code(residual)
    with _on(x, w, bias, residual):
        out = _new(out, shape, x.dtype if out_dtype is None else out_dtype, x.device)
        pre = torch.empty(shape, dtype=torch.float32, device=x.device) if keep_pre else None
        p = LinearParams(_ptr(w), _ptr(bias), _ptr(residual), _dtype_code(x), _dtype_code(w), dtr,
                         _dtype_code(out), code, _stream(stream, x))
        _check(lib().srnl_linear_fwd(_ptr(x), x.numel() // max(K, 1), K, N, ctypes.byref(p), _ptr(out),
                                     _ptr(pre)), "srnl_linear_fwd")
    return (out, pre) if keep_pre else out


def linear_bwd(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
               pre: Optional[torch.Tensor] = None, *, act="none",
               dx_add: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
               need_db: bool = True, stream=None):
    """srnl_linear_bwd: dout [..., N] -> (dx [..., K] in x's dtype, dw [N, K]
    fp32, db [N] fp32), None where not needed (db comes with dw). pre: from
    linear_fwd(keep_pre=True), for an activation. dx_add: a gradient of x's
    shape and dtype, added to dx."""
    N, K = w.shape
    if x.shape[-1] != K:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [..., {K}]")
    shape = x.shape[:-1] + (N,)
    code = _act_code(act)
    _expect(dout, shape, None, "dout")
    _expect(dx_add, x.shape, x.dtype, "dx_add")
    if code == ACT_NONE:
        pre = None
    elif pre is None:
        raise ValueError("an activation's backward needs pre (linear_fwd with keep_pre=True)")
    _expect(pre, shape, torch.float32, "pre")
    if need_db and not need_dw:
        raise ValueError("need_db needs need_dw: the bias gradient is formed with the weight's")
    M = x.numel() // max(K, 1)
    with _on(x, dout, w, pre, dx_add):
        sh = _stream(stream, x)
        p = LinearParams(_ptr(w), None, None, _dtype_code(x), _dtype_code(w), 0,
                         _dtype_code(dout), code, sh)
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty_like(w, dtype=torch.float32) if need_dw else None
        db = torch.empty(N, dtype=torch.float32, device=x.device) if need_db else None
        ws = _workspace(lib().srnl_linear_bwd_workspace_bytes(M, K, N, ctypes.byref(p)), x.device)
        _check(lib().srnl_linear_bwd(_ptr(dout), _ptr(x), M, K, N, ctypes.byref(p), _ptr(pre),
                                     _ptr(dx_add), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws),
                                     0 if ws is None else ws.numel()), "srnl_linear_bwd")
        _keep_for_stream(sh, ws)
    return dx, dw, db


def dwconv_fwd(u: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
               add1: Optional[torch.Tensor] = None, add2: Optional[torch.Tensor] = None, *,
               out_dtype=None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """srnl_dwconv_fwd: the depthwise 3x3 convolution of u [B,H,W,C] (zero
    padding) with w [C,3,3], bias [C] fp32, plus the addends of u's shape, in
    out_dtype (u's when None)."""
    B, H, W, C = u.shape
    _expect(w, (C, 3, 3), torch.float32, "w")
    _expect(bias, (C,), torch.float32, "bias")
    for t, name in ((add1, "add1"), (add2, "add2")):
        _expect(t, u.shape, None, name)
    codes = [0 if t is None else _dtype_code(t) for t in (add1, add2)]
    with _on(u, w, bias, add1, add2):
        out = _new(out, u.shape, u.dtype if out_dtype is None else out_dtype, u.device, like=u)
        _check(lib().srnl_dwconv_fwd(_ptr(u), B, H, W, C, _dtype_code(u), _ptr(w), _ptr(bias),
                                     _ptr(add1), codes[0], _ptr(add2), codes[1], _dtype_code(out),
                                     _ptr(out), _stream(stream, u)), "srnl_dwconv_fwd")
    return out


def dwconv_bwd(dout: torch.Tensor, u: torch.Tensor, w: torch.Tensor, *,
               du_add: Optional[torch.Tensor] = None, need_du: bool = True,
               param_grads: bool = True, stream=None):
    """srnl_dwconv_bwd: dout [B,H,W,C] -> (du in u's dtype, dw [C,3,3], db [C]
    fp32), None where not needed. du_add: another gradient of u, of its shape
    and dtype, added to du."""
    B, H, W, C = u.shape
    _expect(w, (C, 3, 3), torch.float32, "w")
    _expect(dout, u.shape, None, "dout")
    _expect(du_add, u.shape, u.dtype, "du_add")
    with _on(u, dout, w, du_add):
        du = torch.empty_like(u) if need_du else None
        dw = db = ws = None
        if param_grads:
            dw = torch.empty_like(w)
            db = torch.empty(C, dtype=torch.float32, device=u.device)
            ws = _workspace(lib().srnl_dwconv_bwd_workspace_bytes(B, H, W, C), u.device)
        sh = _stream(stream, u)
        _check(lib().srnl_dwconv_bwd(_ptr(dout), _dtype_code(dout), _ptr(u), B, H, W, C,
                                     _dtype_code(u), _ptr(w), _ptr(du_add), _ptr(du), _ptr(dw),
                                     _ptr(db), _ptr(ws), 0 if ws is None else ws.numel(), sh),
               "srnl_dwconv_bwd")
        _keep_for_stream(sh, ws)
    return du, dw, db


def group_norm_fwd(x: torch.Tensor, groups: int, gain: Optional[torch.Tensor],
                   bias: Optional[torch.Tensor], eps: float = 1e-5, *, act="none", out_dtype=None,
                   stats: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """srnl_group_norm_fwd: act of the group norm of x [B, ..., C] (channels
    last, statistics over the cells between and the channels of a group) in
    out_dtype (x's when None); with stats also (mean, rstd) [B, groups] fp32,
    which group_norm_bwd takes. gain, bias: [C] fp32 or None. act as in
    linear_fwd."""
    B, S, C = _map(x)
    for t, name in ((gain, "gain"), (bias, "bias")):
        _expect(t, (C,), torch.float32, name)
    code, dtx = _act_code(act), _dtype_code(x)
    with _on(x, gain, bias):
        out = _new(out, x.shape, x.dtype if out_dtype is None else out_dtype, x.device, like=x)
        dto = _dtype_code(out)
        mean = rstd = None
        if stats:
            mean = torch.empty((B, groups), dtype=torch.float32, device=x.device)
            rstd = torch.empty_like(mean)
        ws = _workspace(lib().srnl_group_norm_fwd_workspace_bytes(B, S, C, groups), x.device)
        sh = _stream(stream, x)
        _check(lib().srnl_group_norm_fwd(_ptr(x), B, S, C, groups, dtx, _ptr(gain), _ptr(bias), eps,
                                         code, dto, _ptr(out), _ptr(mean), _ptr(rstd), _ptr(ws),
                                         0 if ws is None else ws.numel(), sh), "srnl_group_norm_fwd")
        _keep_for_stream(sh, ws)
    return (out, mean, rstd) if stats else out


def group_norm_bwd(dout: torch.Tensor, x: torch.Tensor, groups: int, gain: Optional[torch.Tensor],
                   bias: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor, *,
                   act="none", dx_add: Optional[torch.Tensor] = None, need_dx: bool = True,
                   param_grads: bool = True, stream=None):
    """srnl_group_norm_bwd: dout [B, ..., C] -> (dx in x's dtype, dgain, dbias
    [C] fp32), None where not needed. dx_add: a gradient of x's shape and
    dtype, added to dx."""
    B, S, C = _map(x)
    for t, name in ((gain, "gain"), (bias, "bias")):
        _expect(t, (C,), torch.float32, name)
    _expect(dout, x.shape, None, "dout")
    _expect(dx_add, x.shape, x.dtype, "dx_add")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _expect(t, (B, groups), torch.float32, name)
    code, dtx, dto = _act_code(act), _dtype_code(x), _dtype_code(dout)
    with _on(x, dout, gain, bias, mean, rstd, dx_add):
        dx = torch.empty_like(x) if need_dx else None
        dgain = torch.empty(C, dtype=torch.float32, device=x.device) if param_grads else None
        dbias = torch.empty_like(dgain) if param_grads else None
        ws = _workspace(lib().srnl_group_norm_bwd_workspace_bytes(B, S, C, groups), x.device)
        sh = _stream(stream, x)
        _check(lib().srnl_group_norm_bwd(
            _ptr(dout), dto, _ptr(x), B, S, C, groups, dtx, _ptr(gain), _ptr(bias), _ptr(mean),
            _ptr(rstd), code, _ptr(dx_add), _ptr(dx), _ptr(dgain), _ptr(dbias), _ptr(ws),
            0 if ws is None else ws.numel(), sh), "srnl_group_norm_bwd")
        _keep_for_stream(sh, ws)
    return dx, dgain, dbias


def _map(x: torch.Tensor):
    """(items, cells, channels) of a channels-last map."""
    if x.dim() < 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [B, ..., C]")
    B, C = x.shape[0], x.shape[-1]
    S = 1
    for n in x.shape[1:-1]:
        S *= n
    return B, S, C


_MASK64 = (1 << 64) - 1


def dropout_fwd(x: torch.Tensor, p: float, seed: int, offset: int = 0, *,
                residual: Optional[torch.Tensor] = None, counter: Optional[torch.Tensor] = None,
                out_dtype=None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """srnl_dropout_fwd: x / (1 - p) where kept, else 0, plus the residual of
    x's shape, in out_dtype (x's when None). The mask is a function of seed,
    offset (64 bits each) and the element's place. counter: an int64 tensor of
    one number on x's device, read when the kernel runs and added to offset
    (advance it inside a captured graph, and each replay draws a new mask)."""
    _expect(residual, x.shape, None, "residual")
    _expect(counter, (1,), torch.int64, "counter")
    dtx, dtr = _dtype_code(x), 0 if residual is None else _dtype_code(residual)
    with _on(x, residual, counter):
        out = _new(out, x.shape, x.dtype if out_dtype is None else out_dtype, x.device, like=x)
        _check(lib().srnl_dropout_fwd(_ptr(x), dtx, x.numel(), p, seed & _MASK64, offset & _MASK64,
                                      _ptr(counter), _ptr(residual), dtr, _dtype_code(out),
                                      _ptr(out), _stream(stream, x)), "srnl_dropout_fwd")
    return out


def dropout_bwd(dout: torch.Tensor, p: float, seed: int, offset: int = 0, *, dtype=None,
                dx_add: Optional[torch.Tensor] = None, counter: Optional[torch.Tensor] = None,
                dx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """srnl_dropout_bwd: the gradient of x in dtype (dout's when None), with the
    forward's p, seed, offset and counter. dx_add: a gradient of that shape and
    dtype, added to it."""
    dtype = dout.dtype if dtype is None else dtype
    _expect(dx_add, dout.shape, dtype, "dx_add")
    _expect(counter, (1,), torch.int64, "counter")
    dto = _dtype_code(dout)
    with _on(dout, dx_add, counter):
        dx = _new(dx, dout.shape, dtype, dout.device, "dx", dout)
        _check(lib().srnl_dropout_bwd(_ptr(dout), dto, dout.numel(), p, seed & _MASK64,
                                      offset & _MASK64, _ptr(counter), _ptr(dx_add), _dtype_code(dx),
                                      _ptr(dx), _stream(stream, dout)), "srnl_dropout_bwd")
    return dx


# ---- the gated delta rule

def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements between tokens of t [B, T, heads, D], whose heads must be dense
    and whose items must follow one another (a slice of one projection)."""
    B, T, h, d = t.shape
    if t.is_contiguous():
        return 0
    s = t.stride()
    step = s[1] if T > 1 else s[0]
    # a broadcast token has step 0, which is dense to the library
    if s[3] != 1 or (h > 1 and s[2] != d) or step < h * d or (T > 1 and B > 1 and s[0] != T * step):
        raise ValueError(f"{name} must be contiguous, or a slice of the last axis of a contiguous "
                         "[B, T, ...] tensor (a broadcast one is neither)")
    return step


def _delta_shapes(q, k, v, g, beta, state, lengths):
    """(B, T, Hk, H, Dk, Dv) of a call whose shapes and types agree."""
    if q.dim() != 4 or v.dim() != 4:
        t, name = (q, "q") if q.dim() != 4 else (v, "v")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [B, T, heads, D]")
    B, T, Hk, Dk = q.shape
    _, _, H, Dv = v.shape
    _expect(k, (B, T, Hk, Dk), q.dtype, "k")
    _expect(v, (B, T, H, Dv), q.dtype, "v")
    _expect(g, (B, T, H), torch.float32, "g")
    _expect(beta, (B, T, H), torch.float32, "beta")
    _expect(state, (B, H, Dk, Dv), torch.float32, "state")
    _expect(lengths, (B,), torch.int32, "lengths")
    return B, T, Hk, H, Dk, Dv


def _delta_params(sizes, q, k, v, g, beta, state, lengths, scale, norm_eps, stream):
    return GatedDeltaParams(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), _ptr(beta), _ptr(state), _ptr(lengths),
        *sizes, _token_stride(q, "q"), _token_stride(k, "k"), _token_stride(v, "v"),
        _dtype_code(q), sizes[4] ** -0.5 if scale is None else scale, norm_eps, _stream(stream, q))


def _written(state: Optional[torch.Tensor]) -> None:
    """States go from call to call in one tensor: a graph that holds what was in it
    has to notice, as of torch's own in-place operations."""
    if state is not None:
        torch._C._increment_version((state,))


def gated_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     beta: torch.Tensor, state: torch.Tensor, *, lengths: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None, norm_eps: float = 0.0,
                     state_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     stream=None):
    """srnl_gated_delta_step: a few tokens appended to each sequence, q, k [B, T,
    Hk, Dk], v [B, T, H, Dv], g, beta [B, T, H], lengths [B] int32 or None.
    Returns (out [B, T, H, Dv] in q's dtype, the states after the last token):
    state [B, H, Dk, Dv] itself, updated in place, unless state_out is given.
    scale: 1 / sqrt(Dk) when None. It has no gradient, and raises where autograd
    wants one: gated_delta has."""
    # (_tracked, without its loop's 1.5 us on the host)
    if (torch.is_grad_enabled()
            and (q.requires_grad or k.requires_grad or v.requires_grad or g.requires_grad
                 or beta.requires_grad or (state is not None and state.requires_grad)
                 or (state_out is not None and state_out.requires_grad)
                 or (out is not None and out.requires_grad))
            or forward_ad._current_level >= 0 and _tracked(q, k, v, g, beta, state, state_out, out)):
        raise RuntimeError("gated_delta_step has no gradient: call it under torch.no_grad(), on detached "
                           "tensors, or use gated_delta")
    sizes = _delta_shapes(q, k, v, g, beta, state, lengths)
    with _on(q, k, v, g, beta, state, lengths):
        p = _delta_params(sizes, q, k, v, g, beta, state, lengths, scale, norm_eps, stream)
        state_out = state if state_out is None else _new(state_out, state.shape, torch.float32,
                                                         q.device, "state_out")
        out = _new(out, v.shape, q.dtype, q.device, like=v if v.is_contiguous() else None)
        _check(lib().srnl_gated_delta_step(ctypes.byref(p), _ptr(out), _ptr(state_out)),
               "srnl_gated_delta_step")
    _written(state_out)
    return out, state_out


def gated_delta_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, *, state: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    norm_eps: float = 0.0, record: bool = False,
                    state_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream=None):
    """srnl_gated_delta_fwd: whole sequences, arguments as gated_delta_step's
    (state None: zeros). Returns (out, the states after the last token); with
    record also the record that gated_delta_bwd takes."""
    L = lib()
    sizes = _delta_shapes(q, k, v, g, beta, state, lengths)
    B, T, Hk, H, Dk, Dv = sizes
    with _on(q, k, v, g, beta, state, lengths):
        p = _delta_params(sizes, q, k, v, g, beta, state, lengths, scale, norm_eps, stream)
        state_out = _new(state_out, (B, H, Dk, Dv), torch.float32, q.device, "state_out")
        out = _new(out, v.shape, q.dtype, q.device, like=v if v.is_contiguous() else None)
        rec = None
        if record:
            rec = torch.empty(L.srnl_gated_delta_record_bytes(ctypes.byref(p)), dtype=torch.uint8,
                              device=q.device)
        ws = _workspace(L.srnl_gated_delta_fwd_workspace_bytes(ctypes.byref(p)), q.device)
        _check(L.srnl_gated_delta_fwd(ctypes.byref(p), _ptr(out), _ptr(state_out), _ptr(rec),
                                      0 if rec is None else rec.numel(), _ptr(ws),
                                      0 if ws is None else ws.numel()), "srnl_gated_delta_fwd")
        _keep_for_stream(p.stream, ws)
    _written(state_out)
    return (out, state_out, rec) if record else (out, state_out)


def gated_delta_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    g: torch.Tensor, beta: torch.Tensor, record: torch.Tensor, *,
                    state: Optional[torch.Tensor] = None, dstate: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    norm_eps: float = 0.0, stream=None):
    """srnl_gated_delta_bwd: dout [B, T, H, Dv], record from gated_delta_fwd with
    the same arguments, dstate the gradient of the states it returned (None: 0).
    Returns (dq, dk, dv in q's dtype, dg, dbeta fp32, the gradient of state, or
    None without one)."""
    L = lib()
    sizes = _delta_shapes(q, k, v, g, beta, state, lengths)
    B, T, Hk, H, Dk, Dv = sizes
    _expect(dout, v.shape, q.dtype, "dout")
    _expect(dstate, (B, H, Dk, Dv), torch.float32, "dstate")
    if record.dtype != torch.uint8 or record.dim() != 1:
        raise ValueError("record must be the one that gated_delta_fwd(record=True) returned")
    with _on(q, k, v, g, beta, state, lengths, dout, record, dstate):
        p = _delta_params(sizes, q, k, v, g, beta, state, lengths, scale, norm_eps, stream)
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dk = torch.empty_like(dq)
        dv = torch.empty(v.shape, dtype=q.dtype, device=q.device)
        dg, dbeta = torch.empty_like(g), torch.empty_like(g)
        ds = None if state is None else torch.empty_like(state)
        ws = _workspace(L.srnl_gated_delta_bwd_workspace_bytes(ctypes.byref(p)), q.device)
        _check(L.srnl_gated_delta_bwd(ctypes.byref(p), _ptr(dout), _ptr(dstate), _ptr(record),
                                      record.numel(), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
                                      _ptr(dbeta), _ptr(ds), _ptr(ws),
                                      0 if ws is None else ws.numel()), "srnl_gated_delta_bwd")
        _keep_for_stream(p.stream, ws)
    return dq, dk, dv, dg, dbeta, ds


# ---- the layers as autograd nodes (on the current stream; reverse mode, once
# differentiable: forward-mode tangents and second derivatives raise)

def _dense(dout: torch.Tensor) -> torch.Tensor:
    """An incoming gradient as the entry points take it: contiguous, from a
    16-byte boundary (a slice of a larger gradient may start anywhere)."""
    dout = dout.contiguous()
    return dout.clone() if dout.data_ptr() % 16 else dout


def _tracked(*tensors: Optional[torch.Tensor]) -> bool:
    """Whether autograd has to see the call: a gradient is wanted, or a tensor
    carries a forward-mode tangent (the node has none to give and raises)."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    return forward_ad._current_level >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


class LayerNorm(torch.autograd.Function):
    """srnl_layer_norm_fwd and srnl_layer_norm_bwd as an autograd node."""

    @staticmethod
    def forward(ctx, x, gain, bias, eps, out_dtype):
        out, mean, rstd = layer_norm_fwd(x, gain, bias, eps, out_dtype=out_dtype, stats=True)
        ctx.save_for_backward(x, gain, mean, rstd)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, gain, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dgain, dbias = layer_norm_bwd(_dense(dout), x, gain, mean, rstd,
                                          param_grads=need[1] or need[2])
        return dx, dgain if need[1] else None, dbias if need[2] else None, None, None


def layer_norm(x: torch.Tensor, gain: Optional[torch.Tensor], bias: Optional[torch.Tensor],
               eps: float = 1e-5, out_dtype=None) -> torch.Tensor:
    """Differentiable layer norm over the last axis (layer_norm_fwd)."""
    if not _tracked(x, gain, bias):
        return layer_norm_fwd(x, gain, bias, eps, out_dtype=out_dtype)
    return LayerNorm.apply(x, gain, bias, eps, out_dtype)


class Linear(torch.autograd.Function):
    """srnl_linear_fwd and srnl_linear_bwd as an autograd node. The gradient
    of w comes back in w's dtype (rounded once from fp32)."""

    @staticmethod
    def forward(ctx, x, w, bias, residual, act, out_dtype):
        keep = _act_code(act) != ACT_NONE
        out = linear_fwd(x, w, bias, act=act, residual=residual, out_dtype=out_dtype,
                         keep_pre=keep)
        out, pre = out if keep else (out, None)
        ctx.save_for_backward(x, w, pre)
        ctx.cfg = (act, None if residual is None else residual.dtype)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, w, pre = ctx.saved_tensors
        act, res_dtype = ctx.cfg
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            dx, dw, db = linear_bwd(_dense(dout), x, w, pre, act=act, need_dx=need[0],
                                    need_dw=need[1] or need[2], need_db=need[2])
        dw = dw.to(w.dtype) if need[1] else None
        dres = dout.to(res_dtype) if need[3] else None
        return dx, dw, db, dres, None, None


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *, act="none",
           residual: Optional[torch.Tensor] = None, out_dtype=None) -> torch.Tensor:
    """Differentiable act(x w^T + bias) + residual (linear_fwd)."""
    if not _tracked(x, w, bias, residual):
        return linear_fwd(x, w, bias, act=act, residual=residual, out_dtype=out_dtype)
    return Linear.apply(x, w, bias, residual, act, out_dtype)


class DWConv(torch.autograd.Function):
    """srnl_dwconv_fwd and srnl_dwconv_bwd as an autograd node."""

    @staticmethod
    def forward(ctx, u, w, bias, add1, add2, out_dtype):
        ctx.save_for_backward(u, w)
        ctx.add_dtypes = [None if t is None else t.dtype for t in (add1, add2)]
        return dwconv_fwd(u, w, bias, add1, add2, out_dtype=out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        u, w = ctx.saved_tensors
        need = ctx.needs_input_grad
        du = dw = db = None
        if any(need[:3]):
            du, dw, db = dwconv_bwd(_dense(dout), u, w, need_du=need[0],
                                    param_grads=need[1] or need[2])
        adds = [dout.to(t) if n else None for n, t in zip(need[3:5], ctx.add_dtypes)]
        return (du, dw if need[1] else None, db if need[2] else None, *adds, None)


def dwconv(u: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
           add1: Optional[torch.Tensor] = None, add2: Optional[torch.Tensor] = None, *,
           out_dtype=None) -> torch.Tensor:
    """Differentiable depthwise 3x3 branch with its addends (dwconv_fwd)."""
    if not _tracked(u, w, bias, add1, add2):
        return dwconv_fwd(u, w, bias, add1, add2, out_dtype=out_dtype)
    return DWConv.apply(u, w, bias, add1, add2, out_dtype)


class GroupNorm(torch.autograd.Function):
    """srnl_group_norm_fwd and srnl_group_norm_bwd as an autograd node."""

    @staticmethod
    def forward(ctx, x, groups, gain, bias, eps, act, out_dtype):
        out, mean, rstd = group_norm_fwd(x, groups, gain, bias, eps, act=act, out_dtype=out_dtype,
                                         stats=True)
        ctx.save_for_backward(x, gain, bias, mean, rstd)
        ctx.cfg = (groups, act)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, gain, bias, mean, rstd = ctx.saved_tensors
        groups, act = ctx.cfg
        need = ctx.needs_input_grad
        dx, dgain, dbias = group_norm_bwd(_dense(dout), x, groups, gain, bias, mean, rstd, act=act,
                                          need_dx=need[0], param_grads=need[2] or need[3])
        return (dx, None, dgain if need[2] else None, dbias if need[3] else None, None, None, None)


def group_norm(x: torch.Tensor, groups: int, gain: Optional[torch.Tensor],
               bias: Optional[torch.Tensor], eps: float = 1e-5, *, act="none",
               out_dtype=None) -> torch.Tensor:
    """Differentiable group norm with an activation over x [B, ..., C]
    (group_norm_fwd)."""
    if not _tracked(x, gain, bias):
        return group_norm_fwd(x, groups, gain, bias, eps, act=act, out_dtype=out_dtype)
    return GroupNorm.apply(x, groups, gain, bias, eps, act, out_dtype)


class Dropout(torch.autograd.Function):
    """srnl_dropout_fwd and srnl_dropout_bwd as an autograd node: seed and
    offset are kept, the mask is not. A counter's number is kept too, so that
    it may move on between the passes."""

    @staticmethod
    def forward(ctx, x, p, seed, offset, residual, counter, out_dtype):
        out = dropout_fwd(x, p, seed, offset, residual=residual, counter=counter,
                          out_dtype=out_dtype)
        ctx.save_for_backward(None if counter is None else counter.clone())
        ctx.cfg = (p, seed, offset, x.dtype, None if residual is None else residual.dtype)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        p, seed, offset, dtype, res_dtype = ctx.cfg
        need = ctx.needs_input_grad
        dx = dropout_bwd(_dense(dout), p, seed, offset, dtype=dtype,
                         counter=ctx.saved_tensors[0]) if need[0] else None
        return dx, None, None, None, dout.to(res_dtype) if need[4] else None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, *,
            residual: Optional[torch.Tensor] = None, counter: Optional[torch.Tensor] = None,
            out_dtype=None) -> torch.Tensor:
    """Differentiable dropout, plus the residual (dropout_fwd)."""
    if not _tracked(x, residual):
        return dropout_fwd(x, p, seed, offset, residual=residual, counter=counter,
                           out_dtype=out_dtype)
    return Dropout.apply(x, p, seed, offset, residual, counter, out_dtype)


class GatedDelta(torch.autograd.Function):
    """srnl_gated_delta_fwd and srnl_gated_delta_bwd as an autograd node, with the
    states after the last token as a second output."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, lengths, scale, norm_eps):
        ctx.set_materialize_grads(False)
        out, state_out, record = gated_delta_fwd(q, k, v, g, beta, state=state, lengths=lengths,
                                                 scale=scale, norm_eps=norm_eps, record=True)
        ctx.save_for_backward(q, k, v, g, beta, state, lengths, record)
        ctx.cfg = (scale, norm_eps)
        return out, state_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dstate):
        q, k, v, g, beta, state, lengths, record = ctx.saved_tensors
        scale, norm_eps = ctx.cfg
        dout = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if dout is None else _dense(dout)
        grads = gated_delta_bwd(dout, q, k, v, g, beta, record, state=state,
                                dstate=None if dstate is None else _dense(dstate), lengths=lengths,
                                scale=scale, norm_eps=norm_eps)
        return (*grads, None, None, None)


def gated_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                beta: torch.Tensor, state: Optional[torch.Tensor] = None, *,
                lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                norm_eps: float = 0.0):
    """Differentiable gated delta rule: (out, the states after the last token)
    of gated_delta_fwd, with gradients for q, k, v, g, beta and state."""
    if not _tracked(q, k, v, g, beta, state):
        return gated_delta_fwd(q, k, v, g, beta, state=state, lengths=lengths, scale=scale,
                               norm_eps=norm_eps)
    return GatedDelta.apply(q, k, v, g, beta, state, lengths, scale, norm_eps)


BLOCK_KEYS = ("ln1_w", "ln1_b", "wq", "dw_w", "dw_b", "ln2_w", "ln2_b", "w1", "b1", "w2", "b2")


class Block(torch.autograd.Function):
    """The residual block of srnl_block_fwd in its training form: the layers'
    and the operator's entry points in turn, every activation kept in fp32,
    the gradients of shared inputs added inside the backward calls."""

    @staticmethod
    def forward(ctx, x, states, scales, heads, d, route_mask, ln_eps, kw, *weights):
        ln1_w, ln1_b, wq, dw_w, dw_b, ln2_w, ln2_b, w1, b1, w2, b2 = weights
        B, H, W, C = x.shape
        f32 = torch.float32
        u, m1, r1 = layer_norm_fwd(x, ln1_w, ln1_b, ln_eps, out_dtype=f32, stats=True)
        q = linear_fwd(u, wq)
        y, rec = scan_fwd_record(u, states, heads, d, route_mask, q, **kw)
        s = fuse(y, B, H, W, C, route_mask, scales)
        h = dwconv_fwd(u, dw_w, dw_b, x, s, out_dtype=f32)
        v, m2, r2 = layer_norm_fwd(h, ln2_w, ln2_b, ln_eps, stats=True)
        a, z = linear_fwd(v, w1, b1, act=ACT_GELU, keep_pre=True)
        out = linear_fwd(a, w2, b2, residual=h, out_dtype=x.dtype)
        ctx.save_for_backward(x, states, scales, u, m1, r1, q, y, rec, h, m2, r2, v, a, z, *weights)
        ctx.cfg = (heads, d, route_mask, kw)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, states, scales, u, m1, r1, q, y, rec, h, m2, r2, v, a, z, *weights = ctx.saved_tensors
        ln1_w, ln1_b, wq, dw_w, dw_b, ln2_w, ln2_b, w1, b1, w2, b2 = weights
        heads, d, route_mask, kw = ctx.cfg
        dout = _dense(dout)
        da, gw2, gb2 = linear_bwd(dout, a, w2)
        dv, gw1, gb1 = linear_bwd(da, v, w1, z, act=ACT_GELU)
        dh, gl2w, gl2b = layer_norm_bwd(dv, h, ln2_w, m2, r2, dx_add=dout)
        du, dq, dst, dsc = scan_fuse_bwd(u, states, heads, d, y, scales, dh, route_mask, q,
                                         record=rec, **kw)
        du, gdw, gdb = dwconv_bwd(dh, u, dw_w, du_add=du)
        du, gwq, _ = linear_bwd(dq, u, wq, dx_add=du, need_db=False)
        dx, gl1w, gl1b = layer_norm_bwd(du, x, ln1_w, m1, r1, dx_add=dh)
        grads = (gl1w, gl1b, gwq, gdw, gdb, gl2w, gl2b, gw1, gb1, gw2, gb2)
        return (dx, dst, dsc, None, None, None, None, None,
                *(g.to(t.dtype) for g, t in zip(grads, weights)))


def block(x: torch.Tensor, states: torch.Tensor, scales: torch.Tensor, bw: dict, heads: int,
          d: int, route_mask: int = 15, ln_eps: float = 1e-5, **kw) -> torch.Tensor:
    """Differentiable residual block, x [B,H,W,C] -> [B,H,W,C] in x's dtype:
    the block of block_fwd (any width C = heads * d, any ffn width), with
    gradients for x, the initial states, the scales and every weight. bw: the
    tensors of block_weights (wq, w1, w2 bf16 or fp32, the others fp32). ``kw``
    are the srnl_params fields (alpha_max, eps, chunk_row, chunk_col, flags).
    Runs on the current stream."""
    if "stream" in kw or "q" in kw:
        raise ValueError("block runs on the current stream and forms its own queries")
    C, F = x.shape[-1], bw["w1"].shape[0]
    shapes = {"ln1_w": (C,), "ln1_b": (C,), "wq": (C, C), "dw_w": (C, 3, 3), "dw_b": (C,),
              "ln2_w": (C,), "ln2_b": (C,), "w1": (F, C), "b1": (F,), "w2": (C, F), "b2": (C,)}
    for k, shp in shapes.items():
        _expect(bw[k], shp, None if k in ("wq", "w1", "w2") else torch.float32, k)
    _expect(scales, (4, C), torch.float32, "scales")
    _expect(states, _state_shape(heads, d), torch.float32, "states")
    return Block.apply(x, states, scales, heads, d, route_mask, ln_eps, kw,
                       *(bw[k] for k in BLOCK_KEYS))

"""ctypes binding of libgdpa.so (the C ABI declared in include/gdpa.h).

Argument marshalling only: every step of GDPA runs in the library's CUDA
kernels.  PyTorch provides device memory and the current CUDA stream.  There
is no CPU fallback: if the shared library is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdpa.so")

PHI_IDENTITY, PHI_SILU, PHI_SOFTMAX, PHI_RELU, PHI_GELU = 0, 1, 2, 3, 4
PHI = {"identity": PHI_IDENTITY, "silu": PHI_SILU, "softmax": PHI_SOFTMAX, "relu": PHI_RELU,
       "gelu": PHI_GELU}
DTYPE_F32, DTYPE_BF16 = 0, 1
STATUS = {0: "GDPA_OK", 1: "GDPA_ERR_INVALID_ARG", 2: "GDPA_ERR_UNSUPPORTED",
          3: "GDPA_ERR_CUDA", 4: "GDPA_ERR_TIMEOUT", 5: "GDPA_ERR_WORKSPACE"}

EXPORTED = ("gdpa_fwd_workspace_size", "gdpa_bwd_workspace_size", "gdpa_fwd", "gdpa_bwd",
            "gdpa_workspace_status", "gdpa_fwd_bias", "gdpa_bwd_bias", "gdpa_weight_gen",
            "gdpa_status_string",
            "gdpa_last_launch_count", "gdpa_timing_enable", "gdpa_timing_read")


class Problem(ctypes.Structure):
    """Mirror of gdpa_problem_t."""
    _fields_ = [("B", ctypes.c_int32), ("h", ctypes.c_int32), ("dh", ctypes.c_int32),
                ("m", ctypes.c_int32), ("max_n", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("total_tokens", ctypes.c_int64), ("phi", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class KernelTime(ctypes.Structure):
    """Mirror of gdpa_kernel_time_t."""
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_float)]


class RotarySpec(ctypes.Structure):
    """Mirror of gdpa_rotary_t."""
    _fields_ = [("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("trained_len", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("mscale", ctypes.c_double)]


class Cache(ctypes.Structure):
    """Mirror of gdpa_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page", ctypes.c_int32), ("hk", ctypes.c_int32), ("dh", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class BlockNorm(ctypes.Structure):
    """Mirror of gdpa_block_norm_t."""
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("sigmoid", ctypes.c_int32), ("B", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class GdpaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


_lib = None


def load(path: str = LIB_PATH):
    """Load libgdpa.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libgdpa.so not built at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, sz, pp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Problem)
    lib.gdpa_fwd_workspace_size.argtypes = [pp, ctypes.POINTER(sz)]
    lib.gdpa_bwd_workspace_size.argtypes = [pp, ctypes.POINTER(sz)]
    lib.gdpa_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdpa_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdpa_workspace_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32)]
    lib.gdpa_fwd_bias.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdpa_bwd_bias.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  sz, vp]
    lib.gdpa_status_string.argtypes = [ctypes.c_int]
    lib.gdpa_status_string.restype = ctypes.c_char_p
    lib.gdpa_last_launch_count.restype = ctypes.c_int32
    lib.gdpa_timing_enable.argtypes = [ctypes.c_int32]
    lib.gdpa_timing_enable.restype = ctypes.c_int
    lib.gdpa_timing_read.argtypes = [ctypes.POINTER(KernelTime), ctypes.c_int32]
    lib.gdpa_timing_read.restype = ctypes.c_int32
    lib.gdpa_weight_gen.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, vp, vp, vp,
                                    vp, vp]
    lib.gdpa_weight_gen_bwd_workspace_size.argtypes = [ctypes.c_int32, ctypes.c_int64,
                                                       ctypes.c_int32, ctypes.POINTER(sz)]
    lib.gdpa_weight_gen_bwd_workspace_size.restype = ctypes.c_int
    lib.gdpa_weight_gen_bwd.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, vp, vp,
                                        vp, vp, vp, vp, sz, vp]
    lib.gdpa_weight_gen_bwd.restype = ctypes.c_int
    i32 = ctypes.c_int32
    lib.gdpa_pool_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.gdpa_pool_workspace_size.restype = ctypes.c_int
    lib.gdpa_pool_fwd.argtypes = [i32, i32, i32, i32, ctypes.c_int64, i32, ctypes.c_float, vp, vp,
                                  vp, vp, vp, vp, vp, sz, vp]
    lib.gdpa_pool_fwd.restype = ctypes.c_int
    lib.gdpa_window_workspace_size.argtypes = [i32, i32, i32, ctypes.c_int64, ctypes.POINTER(sz)]
    lib.gdpa_window_workspace_size.restype = ctypes.c_int
    lib.gdpa_window_fwd.argtypes = [i32, i32, i32, ctypes.c_int64, i32, i32, ctypes.c_float, vp,
                                    vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdpa_window_fwd.restype = ctypes.c_int
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.gdpa_pool_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i64, ctypes.POINTER(sz)]
    lib.gdpa_pool_bwd_workspace_size.restype = ctypes.c_int
    lib.gdpa_pool_bwd.argtypes = [i32, i32, i32, i32, i64, i32, f32] + [vp] * 11 + [sz, vp]
    lib.gdpa_pool_bwd.restype = ctypes.c_int
    lib.gdpa_window_bwd_workspace_size.argtypes = [i32, i32, i32, i64, ctypes.POINTER(sz)]
    lib.gdpa_window_bwd_workspace_size.restype = ctypes.c_int
    lib.gdpa_window_bwd.argtypes = [i32, i32, i32, i64, i32, i32, f32] + [vp] * 11 + [sz, vp]
    lib.gdpa_window_bwd.restype = ctypes.c_int
    rp, cp, np_ = (ctypes.POINTER(x) for x in (RotarySpec, Cache, BlockNorm))
    psz = ctypes.POINTER(sz)
    lib.gdpa_rotary.argtypes = [rp, i32, i32, i32, i32, i64, vp, vp, vp, vp, i64, vp, i64, i32, vp]
    lib.gdpa_cache_append.argtypes = [rp, cp, i32, i32, i64, vp, vp, vp, i64, vp, vp, i64, vp, i64,
                                      vp, vp]
    lib.gdpa_chunk_workspace_size.argtypes = [cp, i32, i32, i64, i32, psz]
    lib.gdpa_chunk_fwd.argtypes = [cp, i32, i32, i64, i32, i32, f32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdpa_block_norm_fwd.argtypes = [np_] + [vp] * 9
    lib.gdpa_block_norm_bwd_workspace_size.argtypes = [np_, psz]
    lib.gdpa_block_norm_bwd.argtypes = [np_] + [vp] * 14 + [sz, vp]
    for name in ("rotary", "cache_append", "chunk_workspace_size", "chunk_fwd", "block_norm_fwd",
                 "block_norm_bwd_workspace_size", "block_norm_bwd"):
        getattr(lib, "gdpa_" + name).restype = ctypes.c_int
    for name in EXPORTED[:8]:
        getattr(lib, name).restype = ctypes.c_int
    if path == LIB_PATH:
        _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def problem(B: int, h: int, dh: int, m: int, total_tokens: int, max_n: int, phi, scale: float,
            dtype: torch.dtype) -> Problem:
    phi = PHI[phi] if isinstance(phi, str) else int(phi)
    dt = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}.get(dtype, -1)
    return Problem(B, h, dh, m, max_n, dt, total_tokens, phi, scale)


def problem_for(q: torch.Tensor, k: torch.Tensor, offsets_host, phi, scale: float,
                max_n: Optional[int] = None) -> Problem:
    """Problem of a batch; ``offsets_host`` is a host sequence (for T and max_n)."""
    B, h, m, dh = k.shape
    off = [int(x) for x in offsets_host]
    T = off[-1]
    if max_n is None:
        max_n = max((off[i + 1] - off[i] for i in range(B)), default=0)
    return problem(B, h, dh, m, T, max_n, phi, scale, q.dtype)


def fwd_workspace_bytes(p: Problem) -> int:
    n = ctypes.c_size_t()
    rc = load().gdpa_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n))
    if rc:
        raise GdpaError(rc, "gdpa_fwd_workspace_size")
    return n.value


def bwd_workspace_bytes(p: Problem) -> int:
    n = ctypes.c_size_t()
    rc = load().gdpa_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n))
    if rc:
        raise GdpaError(rc, "gdpa_bwd_workspace_size")
    return n.value


def workspace(nbytes: int, device) -> torch.Tensor:
    """A 256-byte aligned device buffer (torch's caching allocator aligns to 512)."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def fwd(p: Problem, q, offsets, k, v, o=None, lse=None, ws=None, stream=None
        ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Run gdpa_fwd; allocates the outputs/workspace with torch when not given."""
    lib = load()
    if o is None:
        o = torch.empty_like(q)
    if lse is None and p.phi == PHI_SOFTMAX:
        lse = torch.empty((p.h, p.total_tokens), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(fwd_workspace_bytes(p), q.device)
    rc = lib.gdpa_fwd(ctypes.byref(p), _ptr(q), _ptr(offsets), _ptr(k), _ptr(v), _ptr(o),
                      _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_fwd")
    return o, lse


def bwd(p: Problem, q, offsets, k, v, o, lse, dout, dq=None, dk=None, dv=None, ws=None,
        stream=None):
    """Run gdpa_bwd; returns (dq, dk, dv)."""
    lib = load()
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if ws is None:
        ws = workspace(bwd_workspace_bytes(p), q.device)
    rc = lib.gdpa_bwd(ctypes.byref(p), _ptr(q), _ptr(offsets), _ptr(k), _ptr(v), _ptr(o),
                      _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(),
                      _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_bwd")
    return dq, dk, dv


def fwd_bias(p: Problem, q, offsets, k, v, b1=None, b2=None, o=None, lse=None, ws=None,
             stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Run gdpa_fwd_bias: o = phi(s q k^T + b1) v + b2 (fp32 biases b1 [B,h,m],
    b2 [B,h,dh], either may be None)."""
    lib = load()
    if o is None:
        o = torch.empty_like(q)
    if lse is None and p.phi == PHI_SOFTMAX:
        lse = torch.empty((p.h, p.total_tokens), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(fwd_workspace_bytes(p), q.device)
    rc = lib.gdpa_fwd_bias(ctypes.byref(p), _ptr(q), _ptr(offsets), _ptr(k), _ptr(v), _ptr(b1),
                           _ptr(b2), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_fwd_bias")
    return o, lse


def bwd_bias(p: Problem, q, offsets, k, v, b1, b2, o, lse, dout, dq=None, dk=None, dv=None,
             db1=None, db2=None, want_bias_grads=True, ws=None, stream=None):
    """Run gdpa_bwd_bias; returns (dq, dk, dv, db1, db2) (the last two None
    when ``want_bias_grads`` is False and none were given)."""
    lib = load()
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if want_bias_grads:
        B, h, m, dh = k.shape
        db1 = torch.empty((B, h, m), dtype=torch.float32, device=k.device) if db1 is None else db1
        db2 = torch.empty((B, h, dh), dtype=torch.float32, device=k.device) if db2 is None else db2
    if ws is None:
        ws = workspace(bwd_workspace_bytes(p), q.device)
    rc = lib.gdpa_bwd_bias(ctypes.byref(p), _ptr(q), _ptr(offsets), _ptr(k), _ptr(v), _ptr(b1),
                           _ptr(b2), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(db1), _ptr(db2), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_bwd_bias")
    return dq, dk, dv, db1, db2


def weight_gen(w: torch.Tensor, ctx: torch.Tensor, y: Optional[torch.Tensor] = None,
               status_ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Run gdpa_weight_gen: y [B, F] bf16 = ctx [B, C] applied to w [F, C] (fp32)."""
    F, C = w.shape
    B = ctx.shape[0]
    if y is None:
        y = torch.empty((B, F), dtype=torch.bfloat16, device=w.device)
    rc = load().gdpa_weight_gen(B, F, C, _ptr(w), _ptr(ctx), _ptr(y), _ptr(status_ws),
                                _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_weight_gen")
    return y


def weight_gen_bwd(w: torch.Tensor, ctx: torch.Tensor, dy: torch.Tensor, ws=None, stream=None):
    """Run gdpa_weight_gen_bwd; returns (dw [F, C], dctx [B, C]) in fp32."""
    lib = load()
    F, C = w.shape
    B = ctx.shape[0]
    n = ctypes.c_size_t()
    rc = lib.gdpa_weight_gen_bwd_workspace_size(B, F, C, ctypes.byref(n))
    if rc:
        raise GdpaError(rc, "gdpa_weight_gen_bwd_workspace_size")
    if ws is None:
        ws = workspace(n.value, w.device)
    dw = torch.empty((F, C), dtype=torch.float32, device=w.device)
    dctx = torch.empty((B, C), dtype=torch.float32, device=w.device)
    rc = lib.gdpa_weight_gen_bwd(B, F, C, _ptr(w), _ptr(ctx), _ptr(dy), _ptr(dw), _ptr(dctx),
                                 _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_weight_gen_bwd")
    return dw, dctx


def _batch_shape(offsets_host, shape):
    """(B, T, max_n) of a jagged batch: from ``shape`` when given, else from
    the host copy of the offsets."""
    if shape is not None:
        return tuple(int(x) for x in shape)
    off = [int(x) for x in offsets_host]
    B = len(off) - 1
    return B, off[-1], max((off[i + 1] - off[i] for i in range(B)), default=0)


def pool_fwd(seeds: torch.Tensor, offsets, k: torch.Tensor, v: torch.Tensor, scale: float,
             offsets_host, o=None, lse=None, ws=None, stream=None, want_lse=True, shape=None):
    """Run gdpa_pool_fwd (seed-query attention pooling): seeds [h, S, dh],
    jagged k, v [T, h, dh] with device ``offsets`` (host copy ``offsets_host``
    for B, T and max_n, or ``shape`` = (B, T, max_n)); returns
    (o [B, h, S, dh], lse [B, h, S] or None)."""
    lib = load()
    h, S, dh = seeds.shape
    B, T, max_n = _batch_shape(offsets_host, shape)
    if o is None:
        o = torch.empty((B, h, S, dh), dtype=seeds.dtype, device=seeds.device)
    if lse is None and want_lse:
        lse = torch.empty((B, h, S), dtype=torch.float32, device=seeds.device)
    if ws is None:
        n = ctypes.c_size_t()
        rc = lib.gdpa_pool_workspace_size(B, h, dh, S, ctypes.byref(n))
        if rc:
            raise GdpaError(rc, "gdpa_pool_workspace_size")
        ws = workspace(n.value, seeds.device)
    rc = lib.gdpa_pool_fwd(B, h, dh, S, T, max_n, scale, _ptr(seeds), _ptr(offsets), _ptr(k),
                           _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_pool_fwd")
    return o, lse


def window_fwd(q: torch.Tensor, offsets, k: torch.Tensor, v: torch.Tensor, window: int,
               scale: float, offsets_host, o=None, lse=None, ws=None, stream=None,
               want_lse=True, shape=None):
    """Run gdpa_window_fwd (causal sliding-window attention on jagged q, k, v
    [T, h, dh]; B and max_n from ``offsets_host`` or ``shape`` = (B, T, max_n));
    returns (o [T, h, dh], lse [h, T] or None)."""
    lib = load()
    T, h, dh = q.shape
    B, _, max_n = _batch_shape(offsets_host, shape)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((h, T), dtype=torch.float32, device=q.device)
    if ws is None:
        n = ctypes.c_size_t()
        rc = lib.gdpa_window_workspace_size(B, h, dh, T, ctypes.byref(n))
        if rc:
            raise GdpaError(rc, "gdpa_window_workspace_size")
        ws = workspace(n.value, q.device)
    rc = lib.gdpa_window_fwd(B, h, dh, T, max_n, window, scale, _ptr(q), _ptr(offsets), _ptr(k),
                             _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_window_fwd")
    return o, lse


def pool_bwd(seeds: torch.Tensor, offsets, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
             lse: torch.Tensor, dout: torch.Tensor, scale: float, offsets_host, dk=None, dv=None,
             dseeds=None, ws=None, stream=None, shape=None):
    """Run gdpa_pool_bwd: gradients of gdpa_pool_fwd for dout [B, h, S, dh];
    returns (dseeds fp32 [h, S, dh], dk, dv bf16 [T, h, dh])."""
    lib = load()
    h, S, dh = seeds.shape
    B, T, max_n = _batch_shape(offsets_host, shape)
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dseeds is None:
        dseeds = torch.empty((h, S, dh), dtype=torch.float32, device=seeds.device)
    if ws is None:
        n = ctypes.c_size_t()
        rc = lib.gdpa_pool_bwd_workspace_size(B, h, dh, S, T, ctypes.byref(n))
        if rc:
            raise GdpaError(rc, "gdpa_pool_bwd_workspace_size")
        ws = workspace(n.value, seeds.device)
    rc = lib.gdpa_pool_bwd(B, h, dh, S, T, max_n, scale, _ptr(seeds), _ptr(offsets), _ptr(k),
                           _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dseeds), _ptr(dk),
                           _ptr(dv), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_pool_bwd")
    return dseeds, dk, dv


def window_bwd(q: torch.Tensor, offsets, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
               lse: torch.Tensor, dout: torch.Tensor, window: int, scale: float, offsets_host,
               dq=None, dk=None, dv=None, ws=None, stream=None, shape=None):
    """Run gdpa_window_bwd: gradients of gdpa_window_fwd for dout [T, h, dh];
    returns (dq, dk, dv) bf16 [T, h, dh]."""
    lib = load()
    T, h, dh = q.shape
    B, _, max_n = _batch_shape(offsets_host, shape)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if ws is None:
        n = ctypes.c_size_t()
        rc = lib.gdpa_window_bwd_workspace_size(B, h, dh, T, ctypes.byref(n))
        if rc:
            raise GdpaError(rc, "gdpa_window_bwd_workspace_size")
        ws = workspace(n.value, q.device)
    rc = lib.gdpa_window_bwd(B, h, dh, T, max_n, window, scale, _ptr(q), _ptr(offsets), _ptr(k),
                             _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(ws), ws.numel(), _stream(stream))
    if rc:
        raise GdpaError(rc, "gdpa_window_bwd")
    return dq, dk, dv


def _need(ok, where: str, what: str) -> None:
    if not ok:
        raise GdpaError(1, f"{where} ({what})")


def _i32(where: str, name: str, v) -> int:
    """A whole number as a C int32 (ctypes would cut a longer one to its lower bits)."""
    if type(v) is not int:
        v = operator.index(v)
    if v >> 31 not in (0, -1):
        raise GdpaError(1, f"{where} ({name}: 32 bits)")
    return v


def _operand(where, name, t, dtype, shape, dev) -> int:
    """Address of a contiguous tensor of that type and shape on device number `dev`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        raise GdpaError(1, f"{where} ({name}: a contiguous {dtype} tensor {list(shape)} on cuda:{dev})")
    return t.data_ptr()


def _heads(where, name, t, dtype, shape, dev) -> int:
    """A [T, h, dh] tensor whose heads are contiguous; returns its token stride."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        row, head, one = t.stride()
        if one == 1 and (head == shape[2] or shape[1] == 1):
            return row if shape[0] > 1 else shape[1] * shape[2]
    raise GdpaError(1, f"{where} ({name}: {dtype} {list(shape)} on cuda:{dev}, heads contiguous)")


# The current device and its current stream without the Python objects around them (of which a
# call on one token would spend a tenth of its time).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _On:
    """Makes a device current, and `stream` (when given) the stream that allocations
    belong to, for the length of a call; the allocator keeps the call's tensors until that stream
    has passed it."""

    def __init__(self, dev, stream, tensors):
        self.ctx = [torch.cuda.device(dev)]
        self.tensors = tensors if stream is not None else ()
        if stream is not None:
            at = getattr(stream, "device", None)
            if getattr(at, "index", at) not in (None, dev):
                raise GdpaError(1, f"stream of {at} for tensors on cuda:{dev}")
            if not isinstance(stream, torch.cuda.Stream):
                raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
                stream = torch.cuda.ExternalStream(raw, device=dev)
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()
        for t in self.tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(torch.cuda.current_stream())

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


def _elsewhere(where, t, stream, *more) -> Optional[_On]:
    """What a call on `t` (and `more` tensors) and `stream` has to run under; None where it is in force already."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise GdpaError(1, f"{where} (a CUDA tensor)")
    dev = t.get_device()
    return None if stream is None and dev == _current_device() else _On(dev, stream, (t, *more))


def rotary_spec(rot: int, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0,
                trained_len: int = 0, low: float = 1.0, high: float = 32.0,
                mscale: float = 1.0) -> RotarySpec:
    """Rotary settings: ``rot`` rotated elements of a head, pairs (2i, 2i+1) when
    ``interleaved`` else (i, i + rot/2), frequencies base^(-2i/rot) divided by
    ``factor``; with ``trained_len`` only the frequencies that make fewer than
    ``high`` turns within it (fully below ``low`` turns) are."""
    w = "rotary_spec"
    return RotarySpec(_i32(w, "rot", int(rot)), int(bool(interleaved)), _i32(w, "trained_len", int(trained_len)), 0,
                      float(base), float(factor), float(low), float(high), float(mscale))


def rotary(spec: RotarySpec, x: torch.Tensor, offsets=None, kv_len=None, positions=None, out=None,
           inverse: bool = False, stream=None) -> torch.Tensor:
    """Run gdpa_rotary: x [T, h, dh] (bf16 or fp32, heads contiguous, any token
    stride) rotated by ``positions`` [T], or by each token's place in its sample
    (``offsets`` [B+1]; with ``kv_len`` [B] the sample ends at that length).
    ``out`` may be ``x``; rows behind the last sample are left as they were (in a
    new ``out``: not set).  ``inverse`` gives the gradient."""
    w = "gdpa_rotary"
    on = _elsewhere(w, x, stream, offsets, kv_len, positions, out)
    if on:
        with on:
            return rotary(spec, x, offsets, kv_len, positions, out, inverse)
    dt, dev = x.dtype, x.get_device()
    _need(x.dim() == 3 and dt in (torch.bfloat16, torch.float32), w, "x: bf16 or fp32 [T, h, dh]")
    T, h, dh = x.shape
    xs = _heads(w, "x", x, dt, (T, h, dh), dev)
    B, off, kv, pos = 0, None, None, None
    if offsets is not None:
        B = offsets.numel() - 1
        off = _operand(w, "offsets", offsets, torch.int32, (B + 1,), dev)
    if kv_len is not None:
        kv = _operand(w, "kv_len", kv_len, torch.int32, (B,), dev)
    if positions is not None:
        pos = _operand(w, "positions", positions, torch.int32, (T,), dev)
    if out is None:
        out, ys = torch.empty((T, h, dh), dtype=dt, device=x.device), h * dh
    else:
        ys = _heads(w, "out", out, dt, (T, h, dh), dev)
    rc = load().gdpa_rotary(ctypes.byref(spec), DTYPE_BF16 if dt is torch.bfloat16 else DTYPE_F32, B,
                            h, dh, T, off, kv, pos, x.data_ptr(), xs, out.data_ptr(), ys,
                            int(bool(inverse)), _raw_stream(dev))
    if rc:
        raise GdpaError(rc, w)
    return out


def _cache(where, cache_k, cache_v, page_table, B) -> Cache:
    _need(isinstance(cache_k, torch.Tensor) and cache_k.dim() == 4, where,
          "cache_k: [num_pages, hk, page, dh]")
    _need(isinstance(page_table, torch.Tensor) and page_table.dim() == 2, where,
          "page_table: [B, max_pages]")
    shape, dev, width = cache_k.shape, cache_k.get_device(), page_table.shape[1]
    pages, hk, page, dh = shape
    return Cache(_operand(where, "cache_k", cache_k, torch.bfloat16, shape, dev),
                 _operand(where, "cache_v", cache_v, torch.bfloat16, shape, dev),
                 _operand(where, "page_table", page_table, torch.int32, (B, width), dev),
                 pages, width, page, hk, dh, 0)


def cache_append(k: torch.Tensor, v: torch.Tensor, offsets, kv_len, page_table, cache_k, cache_v,
                 spec: Optional[RotarySpec] = None, q=None, q_out=None, status_ws=None,
                 stream=None) -> Optional[torch.Tensor]:
    """Run gdpa_cache_append: rotates (``spec``) and stores the new tokens' keys
    and values k, v [T, hk, dh] in the paged cache [num_pages, hk, page, dh];
    ``kv_len`` [B] counts each sample's tokens with the new ones.  With ``q``
    [T, hq, dh] its rotation is returned (``q_out``)."""
    w = "gdpa_cache_append"
    on = _elsewhere(w, cache_k, stream, k, v, offsets, kv_len, page_table, cache_v, q, q_out, status_ws)
    if on:
        with on:
            return cache_append(k, v, offsets, kv_len, page_table, cache_k, cache_v, spec, q, q_out,
                                status_ws)
    dev = cache_k.get_device()
    _need(isinstance(offsets, torch.Tensor) and offsets.numel() >= 2, w, "offsets: [B + 1]")
    B = offsets.numel() - 1
    c = _cache(w, cache_k, cache_v, page_table, B)
    _, hk, _, dh = cache_k.shape
    off = _operand(w, "offsets", offsets, torch.int32, (B + 1,), dev)
    kv = _operand(w, "kv_len", kv_len, torch.int32, (B,), dev)
    _need(isinstance(k, torch.Tensor) and k.dim() == 3, w, "k: [T, hk, dh]")
    T = k.shape[0]
    ks = _heads(w, "k", k, torch.bfloat16, (T, hk, dh), dev)
    vs = _heads(w, "v", v, torch.bfloat16, (T, hk, dh), dev)
    hq, qs, qp, qo = 0, 0, None, None
    if q is not None:
        _need(isinstance(q, torch.Tensor) and q.dim() == 3, w, "q: [T, hq, dh]")
        hq = q.shape[1]
        qs, qp = _heads(w, "q", q, torch.bfloat16, (T, hq, dh), dev), q.data_ptr()
        if q_out is None:
            q_out = torch.empty((T, hq, dh), dtype=torch.bfloat16, device=cache_k.device)
            qo = q_out.data_ptr()
        else:
            qo = _operand(w, "q_out", q_out, torch.bfloat16, (T, hq, dh), dev)
    else:
        _need(q_out is None, w, "q_out without q")
    if status_ws is not None:
        _need(status_ws.get_device() == dev and status_ws.is_contiguous()
              and status_ws.numel() * status_ws.element_size() >= 256, w,
              "status_ws: 256 bytes on the device")
    rc = load().gdpa_cache_append(None if spec is None else ctypes.byref(spec), ctypes.byref(c),
                                  B, hq, T, off, kv, qp, qs, qo, k.data_ptr(), ks, v.data_ptr(), vs,
                                  _ptr(status_ws), _raw_stream(dev))
    if rc:
        raise GdpaError(rc, w)
    return q_out


def chunk_workspace_bytes(cache: Cache, B: int, hq: int, T: int, max_n: int) -> int:
    """Workspace of a chunk_fwd call on T rows (those behind the last sample, which do not count, among them)."""
    n, w = ctypes.c_size_t(), "gdpa_chunk_workspace_size"
    max_n = _i32(w, "max_n", max_n)
    rc = load().gdpa_chunk_workspace_size(ctypes.byref(cache), B, hq, min(T, B * max_n), max_n, ctypes.byref(n))
    if rc:
        raise GdpaError(rc, w)
    return n.value


@functools.lru_cache(maxsize=256)
def _chunk_workspace(device: int, hk: int, dh: int, hq: int, max_n: int) -> int:
    """What gdpa_chunk_workspace_size says for these sizes (the others do not enter it) on the current device."""
    return chunk_workspace_bytes(Cache(256, 256, 256, 1, 1, 16, hk, dh, 0), 1, hq, 0, max_n)


def chunk_fwd(q: torch.Tensor, offsets, kv_len, page_table, cache_k, cache_v, scale: float,
              max_n: int, window: Optional[int] = None, o=None, lse=None, ws=None,
              want_lse: bool = True, stream=None):
    """Run gdpa_chunk_fwd: attention of the new tokens q [T, hq, dh] over each
    sample's ``kv_len`` cached tokens (its own among them), causal and, with
    ``window``, limited to the last ``window`` tokens; ``max_n`` bounds the new
    tokens of a sample (rows of a padded batch that belong to none do not count, and stay as they were: in a
    new ``o`` not set).  Returns (o [T, hq, dh], lse fp32 [hq, T] or None)."""
    w = "gdpa_chunk_fwd"
    on = _elsewhere(w, q, stream, offsets, kv_len, page_table, cache_k, cache_v, o, lse, ws)
    if on:
        with on:
            return chunk_fwd(q, offsets, kv_len, page_table, cache_k, cache_v, scale, max_n, window, o,
                             lse, ws, want_lse)
    dev = q.get_device()
    _need(q.dim() == 3, w, "q: [T, hq, dh]")
    T, hq, dh = q.shape
    max_n = _i32(w, "max_n", max_n)
    window = 0x7fffffff if window is None else _i32(w, "window", min(window, 0x7fffffff))   # (longer than any history)
    _need(isinstance(offsets, torch.Tensor) and offsets.numel() >= 2, w, "offsets: [B + 1]")
    B = offsets.numel() - 1
    c = _cache(w, cache_k, cache_v, page_table, B)
    hk, cdh = cache_k.shape[1], cache_k.shape[3]
    qp = _operand(w, "q", q, torch.bfloat16, (T, hq, cdh), cache_k.get_device())
    off = _operand(w, "offsets", offsets, torch.int32, (B + 1,), dev)
    kv = _operand(w, "kv_len", kv_len, torch.int32, (B,), dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _operand(w, "o", o, torch.bfloat16, (T, hq, dh), dev)
    if lse is not None:
        _operand(w, "lse", lse, torch.float32, (hq, T), dev)
    elif want_lse:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_chunk_workspace(dev, hk, dh, hq, max_n), q.device)
    else:
        _need(ws.get_device() == dev and ws.dtype is torch.uint8 and ws.is_contiguous(), w,
              "ws: a contiguous uint8 tensor on the device")
    rc = load().gdpa_chunk_fwd(ctypes.byref(c), B, hq, T, max_n, window, scale, qp, off, kv, o.data_ptr(),
                               _ptr(lse), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if rc:
        raise GdpaError(rc, w)
    return o, lse


def _block_norm(where, x, f, gate, w_post, w_pre, offsets, alpha, eps, sigmoid):
    """Checks the operands of a block norm: its description, and the addresses of
    offsets, x, f, gate, w_post, w_pre."""
    dt, dev = x.dtype, x.get_device()
    _need(x.dim() == 2 and dt in (torch.bfloat16, torch.float32), where, "x: bf16 or fp32 [T, d]")
    shape = x.shape
    T, d = shape
    at = [None, _operand(where, "x", x, dt, shape, dev), None, None, None, None]
    if f is not None:
        at[2] = _operand(where, "f", f, dt, shape, dev)
    kind, B = 0, 0
    if gate is not None:
        kind = 1
        if offsets is not None:
            kind, B = 2, offsets.numel() - 1
            at[0] = _operand(where, "offsets", offsets, torch.int32, (B + 1,), dev)
        at[3] = _operand(where, "gate", gate, dt, shape if kind == 1 else (B, d), dev)
    else:
        _need(offsets is None, where, "offsets go with a gate shared by a sample's rows")
    if w_post is not None:
        at[4] = _operand(where, "w_post", w_post, torch.float32, (d,), dev)
    if w_pre is not None:
        at[5] = _operand(where, "w_pre", w_pre, torch.float32, (d,), dev)
    return BlockNorm(T, d, DTYPE_BF16 if dt is torch.bfloat16 else DTYPE_F32, kind, int(bool(sigmoid)),
                     B, alpha, eps, 0), at


def block_norm_fwd(x: torch.Tensor, f=None, gate=None, w_post=None, w_pre=None, offsets=None,
                   alpha: float = 1.0, eps: float = 1e-6, sigmoid: bool = False, y=None, n=None,
                   stream=None):
    """Run gdpa_block_norm_fwd: y = x + alpha * act(gate) * (w_post * f / rms(f)),
    n = w_pre * y / rms(y), on [T, d] rows (bf16 or fp32; weights fp32 [d]).
    ``gate`` [T, d], or with ``offsets`` [B+1] one row [B, d] per sample;
    without ``w_post`` f enters as it is, without ``w_pre`` there is no n, without
    ``f`` y is x.  Returns (y, n)."""
    w = "gdpa_block_norm_fwd"
    on = _elsewhere(w, x, stream, f, gate, w_post, w_pre, offsets, y, n)
    if on:
        with on:
            return block_norm_fwd(x, f, gate, w_post, w_pre, offsets, alpha, eps, sigmoid, y, n)
    p, at = _block_norm(w, x, f, gate, w_post, w_pre, offsets, alpha, eps, sigmoid)
    if f is None:
        _need(y is None, w, "y without f")
    elif y is None:
        y = torch.empty_like(x)
    else:
        _operand(w, "y", y, x.dtype, x.shape, x.get_device())
    if w_pre is None:
        _need(n is None, w, "n without w_pre")
    elif n is None:
        n = torch.empty_like(x)
    else:
        _operand(w, "n", n, x.dtype, x.shape, x.get_device())
    rc = load().gdpa_block_norm_fwd(ctypes.byref(p), *at, _ptr(y), _ptr(n), _raw_stream(x.get_device()))
    if rc:
        raise GdpaError(rc, w)
    return (x if f is None else y), n


def block_norm_bwd(y: torch.Tensor, f=None, gate=None, w_post=None, w_pre=None, dy=None, dn=None,
                   offsets=None, alpha: float = 1.0, eps: float = 1e-6, sigmoid: bool = False,
                   dx=None, df=None, dgate=None, ws=None, stream=None):
    """Run gdpa_block_norm_bwd for dy of y and dn of n (``y``: the forward's y, or
    x where there is no f); returns (dx, df, dgate, dw_post, dw_pre), None where
    there is no such operand.  dgate of a sample gate is fp32 [B, d]."""
    w = "gdpa_block_norm_bwd"
    on = _elsewhere(w, y, stream, f, gate, w_post, w_pre, dy, dn, offsets, dx, df, dgate, ws)
    if on:
        with on:
            return block_norm_bwd(y, f, gate, w_post, w_pre, dy, dn, offsets, alpha, eps, sigmoid, dx,
                                  df, dgate, ws)
    lib = load()
    p, at = _block_norm(w, y, f, gate, w_post, w_pre, offsets, alpha, eps, sigmoid)
    dt, shape, dev = y.dtype, y.shape, y.get_device()
    _need((dn is None) == (w_pre is None), w, "dn goes with w_pre")
    if dy is not None:
        _operand(w, "dy", dy, dt, shape, dev)
    if dn is not None:
        _operand(w, "dn", dn, dt, shape, dev)
    if dx is None:
        dx = torch.empty_like(y)
    else:
        _operand(w, "dx", dx, dt, shape, dev)
    if f is None:
        _need(df is None, w, "df without f")
    elif df is None:
        df = torch.empty_like(y)
    else:
        _operand(w, "df", df, dt, shape, dev)
    if gate is None:
        _need(dgate is None, w, "dgate without a gate")
    else:
        gt = torch.float32 if offsets is not None else dt
        if dgate is None:
            dgate = torch.empty(gate.shape, dtype=gt, device=y.device)
        else:
            _operand(w, "dgate", dgate, gt, gate.shape, dev)
    dw_post, dw_pre = (None if t is None else torch.empty_like(t) for t in (w_post, w_pre))
    n = ctypes.c_size_t()
    rc = lib.gdpa_block_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n))
    if rc:
        raise GdpaError(rc, "gdpa_block_norm_bwd_workspace_size")
    if ws is None:
        ws = workspace(n.value, y.device)
    else:
        _need(ws.get_device() == dev and ws.dtype is torch.uint8 and ws.is_contiguous(), w,
              "ws: a contiguous uint8 tensor on the device")
    rc = lib.gdpa_block_norm_bwd(ctypes.byref(p), *at, _ptr(dy), _ptr(dn), dx.data_ptr(), _ptr(df),
                                 _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), ws.data_ptr(), ws.numel(),
                                 _raw_stream(dev))
    if rc:
        raise GdpaError(rc, w)
    return dx, df, dgate, dw_post, dw_pre


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    """Device-detected status of the last call that used ``ws`` (synchronises)."""
    out = ctypes.c_int32()
    rc = load().gdpa_workspace_status(_ptr(ws), _stream(stream), ctypes.byref(out))
    if rc:
        raise GdpaError(rc, "gdpa_workspace_status")
    return out.value


def last_launch_count() -> int:
    return load().gdpa_last_launch_count()


def status_string(code: int) -> str:
    return load().gdpa_status_string(code).decode()


def timing_enable(on: bool = True) -> None:
    """Bracket every later kernel launch on this thread with CUDA events."""
    rc = load().gdpa_timing_enable(1 if on else 0)
    if rc:
        raise GdpaError(rc, "gdpa_timing_enable")


def timing_read() -> dict:
    """{kernel name: (launches, total ms)} since timing_enable(True); clears."""
    cap = 32
    buf = (KernelTime * cap)()
    n = load().gdpa_timing_read(buf, cap)
    if n < 0:
        raise GdpaError(3, "gdpa_timing_read")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(min(n, cap))}

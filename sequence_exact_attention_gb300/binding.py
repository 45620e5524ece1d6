"""ctypes binding of the C-ABI library (``include/ring_attn.h``).

Argument marshalling only: tensors become device pointers and sizes, the
current torch stream becomes the ``stream`` argument, a non-zero status
becomes ``RingAttnError``. Because the library reads and writes through bare
pointers, every tensor a call passes must have exactly the shape and dtype
the call implies, be contiguous and live on the current CUDA device; the
binding checks that first and raises ``ValueError`` otherwise. Every step of the computation runs in the CUDA
kernels of ``_lib/libringattn.so``; there is no fallback of any kind, and a
missing library raises at the first call.
"""

import contextlib
import ctypes
import functools
import math
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libringattn.so")
LIBRARIES = {"release": LIB_PATH,
             "debug": os.path.join(_HERE, "_lib", "libringattn_debug.so")}

RA_BF16, RA_F32, RA_E4M3 = 0, 1, 2
ORDERS = {"contiguous": 0, "zigzag": 1}
PLAN_COLS = 9
MERGE_MAX_N = 16

# every entry point declared in include/ring_attn.h
EXPORTS = ("ring_attn_fwd", "ring_attn_fwd_ex", "ring_attn_visit_log_len",
           "ring_attn_fwd_varlen", "ring_attn_bwd_varlen", "ring_attn_fwd_ulysses",
           "ring_attn_bwd_ulysses",
           "ring_attn_bwd_workspace", "ring_attn_bwd", "ring_attn_bwd_ex",
           "ring_attn_bwd_noalloc",
           "ring_attn_fwd_window", "ring_attn_fwd_window_varlen",
           "ring_attn_bwd_window_workspace", "ring_attn_bwd_window",
           "ring_attn_bwd_window_varlen",
           "attn_lse_merge", "attn_lse_merge_n",
           "kv4_append", "kv4_read", "kv4_attn_workspace", "kv4_attn", "kv4_evict",
           "paged_append", "paged_append_varlen", "paged_read", "paged_attn_workspace",
           "paged_attn", "paged_attn_varlen",
           "ring_attn_plan",
           "ring_attn_expiry_test", "ring_attn_strerror", "ring_attn_version")

_lib = None
_lib_path = LIB_PATH
_T = None           # torch, imported by the first call that takes tensors


def _import_torch():
    global _T
    import torch
    _T = torch
    return torch


class RingAttnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


def use_library(variant):
    """Select the library the next calls go through: "release" (the default)
    or "debug" (the bounds-checked build, same entry points). Returns the
    variant that was in use."""
    global _lib, _lib_path
    prev = next(k for k, p in LIBRARIES.items() if p == _lib_path)
    if LIBRARIES[variant] != _lib_path:
        _lib_path = LIBRARIES[variant]
        _lib = None
    return prev


def load():
    """Load the selected shared library once; raises if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_lib_path):
        raise RuntimeError(
            f"{_lib_path} is missing: build it with "
            "`python -m sequence_exact_attention_gb300.build` (no CPU fallback)")
    lib = ctypes.CDLL(_lib_path)
    c_int, c_float, vp = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
    ip = ctypes.POINTER(ctypes.c_int)
    lib.ring_attn_fwd.restype = c_int
    lib.ring_attn_fwd.argtypes = [vp, vp, vp, vp, vp] + [c_int] * 7 + [c_float, vp]
    lib.ring_attn_fwd_ex.restype = c_int
    lib.ring_attn_fwd_ex.argtypes = ([vp, vp, vp, vp, vp] + [c_int] * 7 + [c_float]
                                     + [c_int] * 3 + [vp, vp, vp])
    lib.ring_attn_visit_log_len.restype = c_int
    lib.ring_attn_visit_log_len.argtypes = [c_int] * 7 + [ip, ip, ip, ip,
                                                          ctypes.POINTER(ctypes.c_longlong)]
    lib.ring_attn_bwd_workspace.restype = c_int
    lib.ring_attn_bwd_workspace.argtypes = [c_int] * 6 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.ring_attn_bwd.restype = c_int
    lib.ring_attn_bwd.argtypes = ([vp] * 9 + [c_int] * 7 + [c_float, c_int, c_int, vp,
                                                             ctypes.c_size_t, vp, vp])
    lib.ring_attn_bwd_ex.restype = c_int
    lib.ring_attn_bwd_ex.argtypes = ([vp] * 9 + [c_int] * 7 + [c_float, c_int, c_int, vp,
                                                                ctypes.c_size_t, c_int, vp, vp])
    lib.ring_attn_bwd_noalloc.restype = c_int
    lib.ring_attn_bwd_noalloc.argtypes = [vp] * 9 + [c_int] * 7 + [c_float, c_int, c_int, vp, vp]
    lib.ring_attn_fwd_ulysses.restype = c_int
    lib.ring_attn_fwd_ulysses.argtypes = [vp] * 5 + [c_int] * 7 + [c_float, c_int, vp, vp]
    lib.ring_attn_bwd_ulysses.restype = c_int
    lib.ring_attn_bwd_ulysses.argtypes = ([vp] * 9 + [c_int] * 7 + [c_float, c_int, vp,
                                                                    ctypes.c_size_t, vp, vp])
    lib.ring_attn_fwd_varlen.restype = c_int
    lib.ring_attn_fwd_varlen.argtypes = ([vp] * 6 + [c_int] * 8 + [c_float, c_int, c_int,
                                                                   vp, vp])
    lib.ring_attn_bwd_varlen.restype = c_int
    lib.ring_attn_bwd_varlen.argtypes = ([vp] * 10 + [c_int] * 8 + [c_float, c_int, c_int, vp,
                                                                    ctypes.c_size_t, vp, vp])
    lib.ring_attn_fwd_window.restype = c_int
    lib.ring_attn_fwd_window.argtypes = ([vp] * 5 + [c_int] * 8 + [c_float, c_int, c_int, vp, vp])
    lib.ring_attn_fwd_window_varlen.restype = c_int
    lib.ring_attn_fwd_window_varlen.argtypes = ([vp] * 6 + [c_int] * 9 + [c_float, c_int, c_int,
                                                                          vp, vp])
    lib.ring_attn_bwd_window_workspace.restype = c_int
    lib.ring_attn_bwd_window_workspace.argtypes = ([c_int] * 10 +
                                                   [ctypes.POINTER(ctypes.c_size_t)])
    lib.ring_attn_bwd_window.restype = c_int
    lib.ring_attn_bwd_window.argtypes = ([vp] * 9 + [c_int] * 8 + [c_float, c_int, c_int, vp,
                                                                   ctypes.c_size_t, vp, vp])
    lib.ring_attn_bwd_window_varlen.restype = c_int
    lib.ring_attn_bwd_window_varlen.argtypes = ([vp] * 10 + [c_int] * 9 +
                                                [c_float, c_int, c_int, vp, ctypes.c_size_t, vp,
                                                 vp])
    lib.attn_lse_merge.restype = c_int
    lib.attn_lse_merge.argtypes = [vp] * 6 + [c_int] * 5 + [vp]
    lib.attn_lse_merge_n.restype = c_int
    lib.attn_lse_merge_n.argtypes = [vp, vp, c_int, vp, vp] + [c_int] * 5 + [vp]
    lib.kv4_append.restype = c_int
    lib.kv4_append.argtypes = [vp] * 8 + [c_int] * 6 + [vp, vp]
    lib.kv4_read.restype = c_int
    lib.kv4_read.argtypes = [vp] * 7 + [c_int] * 6 + [vp, vp]
    lib.kv4_attn_workspace.restype = c_int
    lib.kv4_attn_workspace.argtypes = [c_int] * 10 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.kv4_attn.restype = c_int
    lib.kv4_attn.argtypes = [vp] * 9 + [c_int] * 9 + [c_float, c_int, vp, ctypes.c_size_t, vp, vp]
    lib.kv4_evict.restype = c_int
    lib.kv4_evict.argtypes = [vp] * 13 + [c_int] * 8 + [vp, vp]
    pages = ctypes.c_char_p          # a struct, as bytes
    lib.paged_append.restype = c_int
    lib.paged_append.argtypes = [pages, vp, c_int] + [vp] * 4 + [c_int] * 3 + [vp, vp]
    lib.paged_append_varlen.restype = c_int
    lib.paged_append_varlen.argtypes = [pages, vp, c_int] + [vp] * 4 + [c_int] * 3 + [vp, vp]
    lib.paged_read.restype = c_int
    lib.paged_read.argtypes = [pages, vp, c_int] + [vp] * 3 + [c_int] * 3 + [vp, vp]
    lib.paged_attn_workspace.restype = c_int
    lib.paged_attn_workspace.argtypes = [pages] + [c_int] * 8 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.paged_attn.restype = c_int
    lib.paged_attn.argtypes = ([vp, pages, vp, c_int] + [vp] * 3 + [c_int] * 6 +
                               [c_float, c_int, vp, ctypes.c_size_t, vp, vp])
    lib.paged_attn_varlen.restype = c_int
    lib.paged_attn_varlen.argtypes = ([vp, pages, vp, c_int] + [vp] * 4 + [c_int] * 7 +
                                      [c_float, c_int, vp, ctypes.c_size_t, vp, vp])
    lib.ring_attn_plan.restype = c_int
    lib.ring_attn_plan.argtypes = [c_int, c_int, c_int, c_int, ip, ctypes.c_size_t]
    lib.ring_attn_expiry_test.restype = c_int
    lib.ring_attn_expiry_test.argtypes = [vp, vp, vp, vp, vp, c_int, vp, vp]
    lib.ring_attn_strerror.restype = ctypes.c_char_p
    lib.ring_attn_strerror.argtypes = [c_int]
    lib.ring_attn_version.restype = c_int
    lib.ring_attn_version.argtypes = []
    _lib = lib
    return lib


def strerror(status):
    return load().ring_attn_strerror(int(status)).decode()


def _check(status, where):
    if status != 0:
        raise RingAttnError(status, where)


# ------------------------------------------------------------------ host-only

def ring_attn_plan(S, P, causal, order="contiguous"):
    """The ring schedule table, int32 [P*P, 9] (see ring_attn_plan in the header)."""
    lib = load()
    n = P * P * PLAN_COLS
    buf = (ctypes.c_int * n)()
    _check(lib.ring_attn_plan(S, P, int(bool(causal)), ORDERS[order], buf, n),
           "ring_attn_plan")
    return np.frombuffer(buf, dtype=np.int32).reshape(P * P, PLAN_COLS).copy()


def visit_log_layout(B, H_q, S, D, P, dtype, order="contiguous"):
    """dict(tile_rows, tiles_per_segment, n_query_tiles, stride, len)."""
    lib = load()
    vals = [ctypes.c_int() for _ in range(4)]
    ln = ctypes.c_longlong()
    _check(lib.ring_attn_visit_log_len(B, H_q, S, D, P, _dtype_code(dtype),
                                       ORDERS[order], *[ctypes.byref(x) for x in vals],
                                       ctypes.byref(ln)), "ring_attn_visit_log_len")
    keys = ("tile_rows", "tiles_per_segment", "n_query_tiles", "stride")
    out = {k: v.value for k, v in zip(keys, vals)}
    out["len"] = ln.value
    return out


# ------------------------------------------------------------------ tensors

def _dtype_code(dt):
    torch = _T or _import_torch()
    if dt is torch.bfloat16 or dt == "bf16":
        return RA_BF16
    if dt is torch.float32 or dt == "f32":
        return RA_F32
    raise ValueError(f"unsupported dtype {dt}")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream):
    """The handle of ``stream``, or of torch's current one (asked for without
    the Stream object that torch.cuda.current_stream() builds: 3 us a call)."""
    if stream is not None:
        return stream.cuda_stream
    c = (_T or _import_torch())._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _like(t, name, shape, dtype):
    """A tensor the library reads or writes through a bare pointer must have
    exactly the shape and dtype the call implies (None: not given)."""
    if t is None:
        return
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _int_buffer(t, name, n):
    """An int32 buffer of at least n elements (None: not given)."""
    if t is None:
        return
    torch = _T or _import_torch()
    if t.dtype != torch.int32 or t.numel() < n:
        raise ValueError(f"{name} must be int32 with at least {n} elements")


def _int32(n):
    """n as a C int that means the same: ctypes drops the bits past 32, and what
    is out of range stays so at its ends (all tokens, too large, negative)."""
    return max(-1, min(int(n), 0x7fffffff))


def _on_device(named):
    """Every tensor on one CUDA device, contiguous, and that device current
    (the library launches on the current device)."""
    torch = _T or _import_torch()
    devs = set()
    for t, n in named:
        if t is not None:
            if not (t.is_cuda and t.is_contiguous()):
                _dev(t, n)
            devs.add(t.get_device())
    if len(devs) > 1:
        raise ValueError("the call's tensors are on several devices: "
                         f"{[f'cuda:{d}' for d in sorted(devs)]}")
    if devs and next(iter(devs)) != torch.cuda.current_device():
        raise ValueError("the call's tensors must be on the current CUDA device")


def ring_attn_fwd(q, k, v, P, causal, scale=None, order="contiguous", step=-1,
                  out=None, lse=None, want_lse=True, visit_log=None,
                  dev_status=None, stream=None):
    """Ring attention of q [B,S,H_q,D], k/v [B,S,H_kv,D] (CUDA tensors).

    Returns (out, lse). bf16 inputs run on the tensor-core kernel, float32 on
    the exact CUDA-core kernel. With ``step`` = t >= 0 only ring step t runs
    and (out, lse) are that step's float32 partial result.
    """
    torch = _T or _import_torch()
    lib = load()
    B, S, H_q, D = q.shape
    H_kv = k.shape[2]
    if k.shape != (B, S, H_kv, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, S, H_kv, D] matching q")
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share a dtype")
    code = _dtype_code(q.dtype)
    out_dtype = torch.float32 if step >= 0 else q.dtype
    _like(out, "out", (B, S, H_q, D), out_dtype)
    _like(lse, "lse", (B, H_q, S), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    if visit_log is not None:
        _int_buffer(visit_log, "visit_log",
                    visit_log_layout(B, H_q, S, D, P, q.dtype, order)["len"])
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"),
                (visit_log, "visit_log"), (dev_status, "dev_status")))
    if out is None:
        out = torch.empty(B, S, H_q, D, device=q.device, dtype=out_dtype)
    if lse is None and (want_lse or step >= 0):
        lse = torch.empty(B, H_q, S, device=q.device, dtype=torch.float32)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                              B, H_q, H_kv, S, D, P, int(bool(causal)), sc,
                              code, ORDERS[order], int(step), _ptr(visit_log),
                              _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_fwd_ex")
    return out, lse


def ring_attn_fwd_plain(q, k, v, out, lse, P, causal, scale=None, stream=None):
    """The plain ``ring_attn_fwd`` entry point (bf16, contiguous order)."""
    torch = _T or _import_torch()
    lib = load()
    B, S, H_q, D = q.shape
    H_kv = k.shape[2]
    _like(k, "k", (B, S, H_kv, D), q.dtype)
    _like(v, "v", (B, S, H_kv, D), q.dtype)
    _like(out, "out", (B, S, H_q, D), q.dtype)
    _like(lse, "lse", (B, H_q, S), torch.float32)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse")))
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                           B, H_q, H_kv, S, D, P, int(bool(causal)), sc,
                           _stream(stream))
    _check(st, "ring_attn_fwd")
    return out, lse


def bwd_workspace_bytes(B, H_q, S, D, P, order="contiguous"):
    """Bytes of device workspace ``ring_attn_bwd`` needs for this shape."""
    lib = load()
    n = ctypes.c_size_t()
    _check(lib.ring_attn_bwd_workspace(B, H_q, S, D, P, ORDERS[order], ctypes.byref(n)),
           "ring_attn_bwd_workspace")
    return n.value


BWD_PREP, BWD_DKDV, BWD_DQ, BWD_ALL = 1, 2, 4, 7


def ring_attn_bwd(q, k, v, out, lse, dout, P, causal, scale=None, order="contiguous",
                  dq=None, dk=None, dv=None, workspace=None, dev_status=None, stream=None,
                  phases=BWD_ALL):
    """Gradients (dq, dk, dv) of ring attention for the upstream gradient dout.

    ``out`` and ``lse`` are the forward's results for the same arguments. All
    tensors are bf16 CUDA tensors (lse float32 [B, H_q, S]). ``workspace``
    (a uint8 CUDA tensor of at least ``bwd_workspace_bytes`` bytes) is
    allocated here when not given; the library itself allocates nothing.
    ``phases`` other than BWD_ALL selects kernels (ring_attn_bwd_ex); a split
    call must reuse the workspace the prep phase filled.
    """
    torch = _T or _import_torch()
    lib = load()
    B, S, H_q, D = q.shape
    H_kv = k.shape[2]
    for t, n in ((k, "k"), (v, "v"), (dk, "dk"), (dv, "dv")):
        _like(t, n, (B, S, H_kv, D), q.dtype)
    for t, n in ((out, "out"), (dout, "dout"), (dq, "dq")):
        _like(t, n, q.shape, q.dtype)
    _like(lse, "lse", (B, H_q, S), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"), (dout, "dout"),
                (dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace"),
                (dev_status, "dev_status")))
    code = _dtype_code(q.dtype)
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    need = bwd_workspace_bytes(B, H_q, S, D, P, order)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
            _ptr(dv), B, H_q, H_kv, S, D, P, int(bool(causal)), sc, code, ORDERS[order],
            _ptr(workspace), workspace.numel() * workspace.element_size())
    if phases == BWD_ALL:
        st = lib.ring_attn_bwd(*args, _ptr(dev_status), _stream(stream))
    else:
        st = lib.ring_attn_bwd_ex(*args, int(phases), _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_bwd")
    return dq, dk, dv


BWD_NOALLOC_MAX_BYTES = 8 << 20
RA_ERR_RANGE = 10
RA_ERR_SCRATCH = 11


def ring_attn_bwd_noalloc(q, k, v, out, lse, dout, P, causal, scale=None, order="contiguous",
                          dq=None, dk=None, dv=None, dev_status=None, stream=None):
    """``ring_attn_bwd`` through the entry point that allocates nothing.

    For callers that cannot allocate device memory (a plugin whose host
    framework owns the memory pool, a path where cudaMalloc may synchronise):
    the library keeps the backward's workspace in its own built-in 8 MiB
    device array. Pass dq, dk, dv to make the whole call allocation-free; when
    omitted they are allocated here, by torch, as for ``ring_attn_bwd``.
    Calls that overlap on the GPU share that array and race: serialise them.
    A problem needing more than ``BWD_NOALLOC_MAX_BYTES`` of workspace raises
    ``RingAttnError`` with status ``RA_ERR_SCRATCH``.
    """
    torch = _T or _import_torch()
    lib = load()
    B, S, H_q, D = q.shape
    H_kv = k.shape[2]
    for t, n in ((k, "k"), (v, "v"), (dk, "dk"), (dv, "dv")):
        _like(t, n, (B, S, H_kv, D), q.dtype)
    for t, n in ((out, "out"), (dout, "dout"), (dq, "dq")):
        _like(t, n, q.shape, q.dtype)
    _like(lse, "lse", (B, H_q, S), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"), (dout, "dout"),
                (dq, "dq"), (dk, "dk"), (dv, "dv"), (dev_status, "dev_status")))
    code = _dtype_code(q.dtype)
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                   _ptr(dq), _ptr(dk), _ptr(dv), B, H_q, H_kv, S, D, P,
                                   int(bool(causal)), sc, code, ORDERS[order],
                                   _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_bwd_noalloc")
    return dq, dk, dv


def _varlen_args(q, k, v, cu_seqlens, max_seqlen):
    torch = _T or _import_torch()
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be a 1-D int32 CUDA tensor")
    total, H_q, D = q.shape
    H_kv = k.shape[1]
    _like(k, "k", (total, H_kv, D), q.dtype)
    _like(v, "v", (total, H_kv, D), q.dtype)
    return total, H_q, H_kv, D, cu_seqlens.numel() - 1, _int32(max_seqlen)


def ring_attn_fwd_varlen(q, k, v, cu_seqlens, max_seqlen, P, causal, scale=None,
                         order="contiguous", out=None, lse=None, dev_status=None,
                         stream=None):
    """Ring attention of packed sequences: q [total,H_q,D], k/v [total,H_kv,D],
    cu_seqlens int32 [n+1] (CUDA). Returns (out [total,H_q,D], lse [H_q,total])."""
    torch = _T or _import_torch()
    lib = load()
    total, H_q, H_kv, D, n, mx = _varlen_args(q, k, v, cu_seqlens, max_seqlen)
    _like(out, "out", q.shape, q.dtype)
    _like(lse, "lse", (H_q, total), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (cu_seqlens, "cu_seqlens"), (out, "out"),
                (lse, "lse"), (dev_status, "dev_status")))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(H_q, total, device=q.device, dtype=torch.float32)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                  _ptr(cu_seqlens), n, total, mx, H_q, H_kv, D, P,
                                  int(bool(causal)), sc, _dtype_code(q.dtype), ORDERS[order],
                                  _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_fwd_varlen")
    return out, lse


def ring_attn_bwd_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, P, causal,
                         scale=None, order="contiguous", workspace=None, dev_status=None,
                         stream=None):
    """Gradients (dq, dk, dv) of ``ring_attn_fwd_varlen`` for the upstream dout."""
    torch = _T or _import_torch()
    lib = load()
    total, H_q, H_kv, D, n, mx = _varlen_args(q, k, v, cu_seqlens, max_seqlen)
    _like(out, "out", q.shape, q.dtype)
    _like(dout, "dout", q.shape, q.dtype)
    _like(lse, "lse", (H_q, total), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    _on_device(((q, "q"), (k, "k"), (v, "v"), (cu_seqlens, "cu_seqlens"), (out, "out"),
                (lse, "lse"), (dout, "dout"), (workspace, "workspace"),
                (dev_status, "dev_status")))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = bwd_workspace_bytes(n, H_q, mx, D, P, order)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                  _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens), n, total, mx,
                                  H_q, H_kv, D, P, int(bool(causal)), sc, _dtype_code(q.dtype),
                                  ORDERS[order], _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_bwd_varlen")
    return dq, dk, dv


def ring_attn_fwd_ulysses(q, k, v, S, causal, scale=None, out=None, lse=None,
                          dev_status=None, stream=None):
    """Attention of sequence-sharded tensors q [P,B,C,H_q,D], k/v [P,B,C,H_kv,D]
    (C = ceil(S/P)). Returns (out [P,B,C,H_q,D], lse [P,B,H_q,C])."""
    torch = _T or _import_torch()
    lib = load()
    P, B, C, H_q, D = q.shape
    H_kv = k.shape[3]
    _like(k, "k", (P, B, C, H_kv, D), q.dtype)
    _like(v, "v", (P, B, C, H_kv, D), q.dtype)
    if C != -(-S // P):
        raise ValueError("shard length must be ceil(S / P)")
    _like(out, "out", q.shape, q.dtype)
    _like(lse, "lse", (P, B, H_q, C), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"),
                (dev_status, "dev_status")))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(P, B, H_q, C, device=q.device, dtype=torch.float32)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_fwd_ulysses(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv,
                                   S, D, P, int(bool(causal)), sc, _dtype_code(q.dtype),
                                   _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_fwd_ulysses")
    return out, lse


def ring_attn_bwd_ulysses(q, k, v, out, lse, dout, S, causal, scale=None, workspace=None,
                          dev_status=None, stream=None):
    """Gradients (dq, dk, dv) of ``ring_attn_fwd_ulysses``, all in the
    sequence-parallel layout [P, B, C, H, D]."""
    torch = _T or _import_torch()
    lib = load()
    P, B, C, H_q, D = q.shape
    H_kv = k.shape[3]
    _like(k, "k", (P, B, C, H_kv, D), q.dtype)
    _like(v, "v", (P, B, C, H_kv, D), q.dtype)
    if C != -(-S // P):
        raise ValueError("shard length must be ceil(S / P)")
    _like(out, "out", q.shape, q.dtype)
    _like(dout, "dout", q.shape, q.dtype)
    _like(lse, "lse", (P, B, H_q, C), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"), (dout, "dout"),
                (workspace, "workspace"), (dev_status, "dev_status")))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = bwd_workspace_bytes(B, H_q, S, D, P, "contiguous")
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_bwd_ulysses(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                   _ptr(dq), _ptr(dk), _ptr(dv), B, H_q, H_kv, S, D, P,
                                   int(bool(causal)), sc, _dtype_code(q.dtype), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_bwd_ulysses")
    return dq, dk, dv


_NULL_CONTEXT = contextlib.nullcontext()


def _on_stream(stream):
    """Memory handed out inside belongs to the stream the call runs on."""
    if stream is None:
        return _NULL_CONTEXT
    torch = _T or _import_torch()
    return torch.cuda.stream(stream)


def ring_attn_fwd_window(q, k, v, P, window, n_sink=0, scale=None, order="contiguous", out=None,
                         lse=None, want_lse=True, dev_status=None, stream=None):
    """Causal ring attention in which query i sees the ``window`` tokens up to
    itself and the first ``n_sink`` tokens; q [B,S,H_q,D], k/v [B,S,H_kv,D],
    bf16 or float32. Returns (out, lse)."""
    torch = _T or _import_torch()
    lib = load()
    B, S, H_q, D = q.shape
    H_kv = k.shape[2]
    _like(k, "k", (B, S, H_kv, D), q.dtype)
    _like(v, "v", (B, S, H_kv, D), q.dtype)
    _like(out, "out", q.shape, q.dtype)
    _like(lse, "lse", (B, H_q, S), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    code = _dtype_code(q.dtype)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"),
                (dev_status, "dev_status")))
    with _on_stream(stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None and want_lse:
            lse = torch.empty(B, H_q, S, device=q.device, dtype=torch.float32)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, S,
                                  D, _int32(P), _int32(window), _int32(n_sink), sc, code,
                                  ORDERS[order], _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_fwd_window")
    return out, lse


def ring_attn_fwd_window_varlen(q, k, v, cu_seqlens, max_seqlen, P, window, n_sink=0, scale=None,
                                order="contiguous", out=None, lse=None, dev_status=None,
                                stream=None):
    """``ring_attn_fwd_window`` of packed sequences: q [total,H_q,D], k/v
    [total,H_kv,D], cu_seqlens int32 [n+1] (CUDA); windows and first tokens
    are each sequence's own. Returns (out [total,H_q,D], lse [H_q,total])."""
    torch = _T or _import_torch()
    lib = load()
    total, H_q, H_kv, D, n, mx = _varlen_args(q, k, v, cu_seqlens, max_seqlen)
    _like(out, "out", q.shape, q.dtype)
    _like(lse, "lse", (H_q, total), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    code = _dtype_code(q.dtype)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (cu_seqlens, "cu_seqlens"), (out, "out"),
                (lse, "lse"), (dev_status, "dev_status")))
    with _on_stream(stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty(H_q, total, device=q.device, dtype=torch.float32)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_fwd_window_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                         _ptr(cu_seqlens), n, total, mx, H_q, H_kv, D, _int32(P),
                                         _int32(window), _int32(n_sink), sc, code, ORDERS[order],
                                         _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_fwd_window_varlen")
    return out, lse


def bwd_window_workspace_bytes(B, H_q, H_kv, S, D, P, window, n_sink=0, order="contiguous",
                               varlen=False):
    """Bytes of device workspace ``ring_attn_bwd_window`` needs (packed: B
    sequences of at most S tokens, ``varlen``)."""
    lib = load()
    n = ctypes.c_size_t()
    sizes = map(_int32, (B, H_q, H_kv, S, D, P, window, n_sink))
    _check(lib.ring_attn_bwd_window_workspace(*sizes, ORDERS[order], int(bool(varlen)),
                                              ctypes.byref(n)),
           "ring_attn_bwd_window_workspace")
    return n.value


def ring_attn_bwd_window(q, k, v, out, lse, dout, P, window, n_sink=0, scale=None,
                         order="contiguous", dq=None, dk=None, dv=None, workspace=None,
                         dev_status=None, stream=None):
    """Gradients (dq, dk, dv) of ``ring_attn_fwd_window`` (bf16) for the
    upstream dout; ``workspace`` (uint8, ``bwd_window_workspace_bytes``) is
    allocated here when not given."""
    torch = _T or _import_torch()
    lib = load()
    B, S, H_q, D = q.shape
    H_kv = k.shape[2]
    for t, n in ((k, "k"), (v, "v"), (dk, "dk"), (dv, "dv")):
        _like(t, n, (B, S, H_kv, D), q.dtype)
    for t, n in ((out, "out"), (dout, "dout"), (dq, "dq")):
        _like(t, n, q.shape, q.dtype)
    _like(lse, "lse", (B, H_q, S), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    code = _dtype_code(q.dtype)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"), (dout, "dout"),
                (dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace"),
                (dev_status, "dev_status")))
    with _on_stream(stream):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if workspace is None:
            need = bwd_window_workspace_bytes(B, H_q, H_kv, S, D, P, window, n_sink, order)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                  _ptr(dq), _ptr(dk), _ptr(dv), B, H_q, H_kv, S, D, _int32(P),
                                  _int32(window), _int32(n_sink), sc, code, ORDERS[order],
                                  _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                  _stream(stream))
    _check(st, "ring_attn_bwd_window")
    return dq, dk, dv


def ring_attn_bwd_window_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, P, window,
                                n_sink=0, scale=None, order="contiguous", dq=None, dk=None,
                                dv=None, workspace=None, dev_status=None, stream=None):
    """Gradients (dq, dk, dv) of ``ring_attn_fwd_window_varlen`` for the
    upstream dout."""
    torch = _T or _import_torch()
    lib = load()
    total, H_q, H_kv, D, n, mx = _varlen_args(q, k, v, cu_seqlens, max_seqlen)
    for t, name in ((out, "out"), (dout, "dout"), (dq, "dq")):
        _like(t, name, q.shape, q.dtype)
    for t, name in ((dk, "dk"), (dv, "dv")):
        _like(t, name, k.shape, q.dtype)
    _like(lse, "lse", (H_q, total), torch.float32)
    _int_buffer(dev_status, "dev_status", 1)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    code = _dtype_code(q.dtype)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (cu_seqlens, "cu_seqlens"), (out, "out"),
                (lse, "lse"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv"),
                (workspace, "workspace"), (dev_status, "dev_status")))
    with _on_stream(stream):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if workspace is None:
            need = bwd_window_workspace_bytes(n, H_q, H_kv, mx, D, P, window, n_sink, order, True)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(D)
    st = lib.ring_attn_bwd_window_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                         _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                         _ptr(cu_seqlens), n, total, mx, H_q, H_kv, D, _int32(P),
                                         _int32(window), _int32(n_sink), sc, code, ORDERS[order],
                                         _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                         _stream(stream))
    _check(st, "ring_attn_bwd_window_varlen")
    return dq, dk, dv


def attn_lse_merge(o_a, lse_a, o_b, lse_b, out=None, lse=None, stream=None):
    """Pairwise merge; o_* [B,S,H,D], lse_* [B,H,S] float32."""
    torch = _T or _import_torch()
    lib = load()
    B, S, H, D = o_a.shape
    for t, n in ((o_b, "o_b"), (out, "out")):
        _like(t, n, o_a.shape, o_a.dtype)
    for t, n in ((lse_a, "lse_a"), (lse_b, "lse_b"), (lse, "lse")):
        _like(t, n, (B, H, S), torch.float32)
    _on_device(((o_a, "o_a"), (o_b, "o_b"), (lse_a, "lse_a"), (lse_b, "lse_b"), (out, "out"),
                (lse, "lse")))
    if out is None:
        out = torch.empty_like(o_a)
    if lse is None:
        lse = torch.empty_like(lse_a)
    st = lib.attn_lse_merge(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b),
                            _ptr(out), _ptr(lse), B, H, S, D,
                            _dtype_code(o_a.dtype), _stream(stream))
    _check(st, "attn_lse_merge")
    return out, lse


def attn_lse_merge_n(os_, lses, out=None, lse=None, stream=None):
    """N-way merge of lists of partials (one pass)."""
    torch = _T or _import_torch()
    lib = load()
    n = len(os_)
    if n < 1 or len(lses) != n:
        raise ValueError("need as many lse tensors as partial outputs, at least one")
    B, S, H, D = os_[0].shape
    for i, t in enumerate(os_):
        _like(t, f"partial {i}", os_[0].shape, os_[0].dtype)
    for i, t in enumerate(lses):
        _like(t, f"lse {i}", (B, H, S), torch.float32)
    _like(out, "out", os_[0].shape, os_[0].dtype)
    _like(lse, "lse", (B, H, S), torch.float32)
    _on_device([(t, "partial") for t in os_] + [(t, "lse") for t in lses] +
               [(out, "out"), (lse, "lse")])
    if out is None:
        out = torch.empty_like(os_[0])
    if lse is None:
        lse = torch.empty_like(lses[0])
    o_arr = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in os_])
    l_arr = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in lses])
    st = lib.attn_lse_merge_n(o_arr, l_arr, n, _ptr(out), _ptr(lse), B, H, S, D,
                              _dtype_code(os_[0].dtype), _stream(stream))
    _check(st, "attn_lse_merge_n")
    return out, lse


# ------------------------------------------------------------------ 4-bit key/value cache

class KV4Cache(tuple):
    """A key/value cache held in 4 bits (format: ``include/ring_attn.h``):
    codes uint8 [B, H_kv, C, D/2], meta bfloat16 [B, H_kv, C, D/64, 2].

    A tuple of its four tensors, whose shapes, dtypes and layout are checked
    here, once, and not again by the calls that take the cache.
    """
    fields = ("k_codes", "k_meta", "v_codes", "v_meta")

    def __new__(cls, k_codes, k_meta, v_codes, v_meta):
        torch = _T or _import_torch()
        self = super().__new__(cls, (k_codes, k_meta, v_codes, v_meta))
        shape = k_codes.shape
        if len(shape) != 4:
            raise ValueError("k_codes must be [B, H_kv, C, D/2]")
        B, H_kv, C, half = shape
        meta = (B, H_kv, C, half // 32, 2)
        _like(k_codes, "k_codes", shape, torch.uint8)
        _like(v_codes, "v_codes", shape, torch.uint8)
        _like(k_meta, "k_meta", meta, torch.bfloat16)
        _like(v_meta, "v_meta", meta, torch.bfloat16)
        self.dims = (B, H_kv, C, 2 * half)
        self.device = dev = k_codes.get_device()
        for t, n in zip(self, cls.fields):
            if not t.is_contiguous():
                raise ValueError(f"{n} must be contiguous")
            if t.get_device() != dev:
                raise ValueError("the cache's tensors are on several devices")
        return self

    k_codes = property(lambda self: self[0])
    k_meta = property(lambda self: self[1])
    v_codes = property(lambda self: self[2])
    v_meta = property(lambda self: self[3])

    def pointers(self):
        return self[0].data_ptr(), self[1].data_ptr(), self[2].data_ptr(), self[3].data_ptr()


def kv4_cache(B, H_kv, C, D, device="cuda"):
    """A zeroed cache of capacity C (a multiple of 16) slots a sequence."""
    torch = _T or _import_torch()
    if D not in (64, 128) or C <= 0 or C % 16:
        raise ValueError("D must be 64 or 128 and C a positive multiple of 16")
    parts = []
    for _ in range(2):
        parts.append(torch.zeros(B, H_kv, C, D // 2, dtype=torch.uint8, device=device))
        parts.append(torch.zeros(B, H_kv, C, D // 64, 2, dtype=torch.bfloat16, device=device))
    return KV4Cache(*parts)


def _with_cache(cache, tensors, names):
    """The call's other tensors (None: not given) contiguous and on the
    cache's device, and that device current."""
    dev = cache.device
    if dev < 0:
        raise ValueError("the cache must be of CUDA tensors")
    for i, t in enumerate(tensors):
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            _dev(t, names[i])
            raise ValueError(f"{names[i]} and the cache are on different devices")
    if dev != _T._C._cuda_getDevice():
        raise ValueError("the call's tensors must be on the current CUDA device")


def _ints(t, name, n):
    """A contiguous int32 [n] tensor (None: not given)."""
    if t is not None:
        _like(t, name, (n,), (_T or _import_torch()).int32)


def kv4_append(cache, k, v, start, n_new=None, dev_status=None, stream=None):
    """Quantises k, v [B, T, H_kv, D] (bf16 or float32) into slots start[b],
    start[b] + 1, ... of ``cache``; with ``n_new`` int32 [B] only the first
    n_new[b] tokens of a padded batch. start: int32 [B] (CUDA)."""
    lib = load()
    B, H_kv, C, D = cache.dims
    if k.dim() != 4:
        raise ValueError("k must be [B, T, H_kv, D]")
    T = k.shape[1]
    shape = (B, T, H_kv, D)
    _like(k, "k", shape, k.dtype)
    _like(v, "v", shape, k.dtype)
    _ints(start, "start", B)
    _ints(n_new, "n_new", B)
    _int_buffer(dev_status, "dev_status", 1)
    code = _dtype_code(k.dtype)
    _with_cache(cache, (k, v, start, n_new, dev_status), ("k", "v", "start", "n_new", "dev_status"))
    st = lib.kv4_append(k.data_ptr(), v.data_ptr(), *cache.pointers(), start.data_ptr(), _ptr(n_new), B, T, H_kv,
                        D, C, code, _ptr(dev_status), _stream(stream))
    _check(st, "kv4_append")


def kv4_read(cache, start, T, dtype=None, k=None, v=None, dev_status=None, stream=None):
    """The values (k, v) [B, T, H_kv, D] of slots start[b] ... start[b] + T - 1
    (start None: from slot 0), bf16 unless ``dtype`` or a given k or v says
    float32."""
    torch = _T or _import_torch()
    lib = load()
    B, H_kv, C, D = cache.dims
    if dtype is None:
        given = k if k is not None else v
        dtype = torch.bfloat16 if given is None else given.dtype
    code = _dtype_code(dtype)
    T = int(T)
    if T <= 0:
        raise ValueError("T must be positive")
    shape = (B, T, H_kv, D)
    _like(k, "k", shape, dtype)
    _like(v, "v", shape, dtype)
    _ints(start, "start", B)
    _int_buffer(dev_status, "dev_status", 1)
    _with_cache(cache, (k, v, start, dev_status), ("k", "v", "start", "dev_status"))
    with _on_stream(stream):
        if k is None:
            k = torch.empty(shape, dtype=dtype, device=cache[0].device)
        if v is None:
            v = torch.empty(shape, dtype=dtype, device=cache[0].device)
    st = lib.kv4_read(*cache.pointers(), _ptr(start), k.data_ptr(), v.data_ptr(), B, T, H_kv, D, C, code,
                      _ptr(dev_status), _stream(stream))
    _check(st, "kv4_read")
    return k, v


# (a function of the sizes alone; asking the library costs as much as a launch)
@functools.lru_cache(maxsize=256)
def kv4_attn_workspace_bytes(B, S_q, H_q, H_kv, D, C, max_len=None, window=0, n_sink=0,
                             with_score=False):
    """Bytes of device workspace ``kv4_attn`` needs for these sizes."""
    n = ctypes.c_size_t()
    sizes = map(_int32, (B, S_q, H_q, H_kv, D, C, C if max_len is None else max_len, window, n_sink))
    _check(load().kv4_attn_workspace(*sizes, 1 if with_score else 0, ctypes.byref(n)),
           "kv4_attn_workspace")
    return n.value


def kv4_attn(q, cache, lens, max_len=None, window=0, n_sink=0, scale=None, out=None, lse=None,
             score=None, workspace=None, dev_status=None, stream=None):
    """Attention of new tokens q [B, S_q, H_q, D] (bf16) over a 4-bit cache.

    ``lens`` int32 [B] (CUDA) counts the slots in use, the S_q new tokens'
    included; ``max_len`` (default: the capacity) bounds it and sizes the
    launch. ``window`` > 0 limits every query to its last ``window`` slots and
    the first ``n_sink``. ``score`` float32 [B, H_kv, C]: every slot's weight
    is added to it. Returns (out [B, S_q, H_q, D], lse [B, H_q, S_q]). A
    ``workspace`` (uint8, ``kv4_attn_workspace_bytes``) is allocated here when
    not given; calls that may overlap need their own.
    """
    torch = _T or _import_torch()
    lib = load()
    B, H_kv, C, D = cache.dims
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != D:
        raise ValueError("q must be [B, S_q, H_q, D] matching the cache")
    _, S_q, H_q, _ = shape
    max_len = C if max_len is None else _int32(max_len)
    window, n_sink = _int32(window), _int32(n_sink)
    _like(out, "out", shape, q.dtype)
    _like(lse, "lse", (B, H_q, S_q), torch.float32)
    _like(score, "score", (B, H_kv, C), torch.float32)
    _ints(lens, "lens", B)
    _int_buffer(dev_status, "dev_status", 1)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    code = _dtype_code(q.dtype)
    _with_cache(cache, (q, lens, out, lse, score, workspace, dev_status),
                ("q", "lens", "out", "lse", "score", "workspace", "dev_status"))
    with _on_stream(stream):
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((B, H_q, S_q), dtype=torch.float32, device=q.device)
        if workspace is None:
            need = kv4_attn_workspace_bytes(B, S_q, H_q, H_kv, D, C, max_len, window, n_sink,
                                            score is not None)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = lib.kv4_attn(q.data_ptr(), *cache.pointers(), lens.data_ptr(), out.data_ptr(),
                      lse.data_ptr(), _ptr(score), B, S_q, H_q, H_kv, D, C, max_len, window, n_sink,
                      0.0 if scale is None else float(scale), code, _ptr(workspace),
                      0 if workspace is None else workspace.numel(), _ptr(dev_status),
                      _stream(stream))
    _check(st, "kv4_attn")
    return out, lse


def kv4_evict(cache, score, lens, budget, n_sink=0, n_recent=0, dst=None, dst_score=None,
              dst_lens=None, kept=None, dev_status=None, stream=None):
    """Keeps at most ``budget`` slots a sequence and head: the first
    ``n_sink``, the last ``n_recent`` and the largest ``score`` float32
    [B, H_kv, C] between them (ties: the lowest slot), in their order.

    Returns (dst, dst_score, dst_lens, kept): another cache (of capacity
    ``budget`` rounded up to 16 unless given; it may not share memory with
    ``cache``), its scores, its lens int32 [B], and kept int32
    [B, H_kv, budget], every kept slot's place in ``cache`` (-1 past the last).
    Slots of ``dst`` past the last are left as they were.
    """
    torch = _T or _import_torch()
    lib = load()
    B, H_kv, C, D = cache.dims
    budget, n_sink, n_recent = int(budget), _int32(n_sink), _int32(n_recent)
    if budget <= 0:
        raise ValueError("budget must be positive")
    C_dst = -(-budget // 16) * 16
    if dst is not None:
        dB, dH, C_dst, dD = dst.dims
        if (dB, dH, dD) != (B, H_kv, D):
            raise ValueError("dst must have the cache's B, H_kv and D")
    if budget > min(C_dst, 0x7fffffff):
        _check(RA_ERR_RANGE, "kv4_evict")
    _like(score, "score", (B, H_kv, C), torch.float32)
    _like(dst_score, "dst_score", (B, H_kv, C_dst), torch.float32)
    _like(kept, "kept", (B, H_kv, budget), torch.int32)
    _ints(lens, "lens", B)
    _ints(dst_lens, "dst_lens", B)
    _int_buffer(dev_status, "dev_status", 1)
    _with_cache(cache, (score, lens, dst_score, dst_lens, kept, dev_status),
                ("score", "lens", "dst_score", "dst_lens", "kept", "dev_status"))
    if dst is not None and dst.device != cache.device:
        raise ValueError("dst and the cache are on different devices")
    dev = cache[0].device
    with _on_stream(stream):
        if dst is None:
            dst = kv4_cache(B, H_kv, C_dst, D, dev)
        if dst_score is None:
            dst_score = torch.zeros((B, H_kv, C_dst), dtype=torch.float32, device=dev)
        if dst_lens is None:
            dst_lens = torch.empty_like(lens)
        if kept is None:
            kept = torch.empty((B, H_kv, budget), dtype=torch.int32, device=dev)
    st = lib.kv4_evict(*cache.pointers(), _ptr(score), _ptr(lens), *dst.pointers(),
                       _ptr(dst_score), _ptr(dst_lens), _ptr(kept), B, H_kv, D, C, C_dst, budget,
                       n_sink, n_recent, _ptr(dev_status), _stream(stream))
    _check(st, "kv4_evict")
    return dst, dst_score, dst_lens, kept


# ------------------------------------------------------------------ paged key/value cache

# ra_pages of include/ring_attn.h, as bytes
_PAGES = struct.Struct("4P5i")


def _pages(ptrs, dims, quant):
    if quant:
        return _PAGES.pack(*ptrs, *dims, RA_E4M3)
    return _PAGES.pack(*ptrs, 0, 0, *dims, RA_BF16)


class PagedCache(tuple):
    """A pool of pages of keys and values (format: ``include/ring_attn.h``):
    k and v [n_pages, H_kv, page, D], bfloat16 or float8_e4m3fn, the latter with
    k_scale and v_scale uint8 [n_pages, H_kv, page].

    A tuple of its tensors, whose shapes, dtypes and layout are checked here,
    once, and not again by the calls that take the cache: memory behind them may
    be given back and taken again in between, their shapes stay.
    """

    def __new__(cls, k, v, k_scale=None, v_scale=None):
        torch = _T or _import_torch()
        shape, dtype, dev = k.shape, k.dtype, k.get_device()
        quant = dtype is torch.float8_e4m3fn
        if not quant and dtype is not torch.bfloat16:
            raise ValueError(f"pages must be bfloat16 or float8_e4m3fn, got {dtype}")
        if len(shape) != 4:
            raise ValueError("k must be [n_pages, H_kv, page, D]")
        if quant != (k_scale is not None) or quant != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to pages of 8 bits")
        _like(v, "v", shape, dtype)
        parts = (k, v)
        if quant:
            _like(k_scale, "k_scale", shape[:3], torch.uint8)
            _like(v_scale, "v_scale", shape[:3], torch.uint8)
            parts = (k, v, k_scale, v_scale)
        for i, t in enumerate(parts):
            if not t.is_contiguous():
                raise ValueError(f"{('k', 'v', 'k_scale', 'v_scale')[i]} must be contiguous")
            if t.get_device() != dev:
                raise ValueError("the cache's tensors are on several devices")
        if max(shape) > 0x7fffffff:
            _check(RA_ERR_RANGE, "PagedCache")
        self = super().__new__(cls, parts)
        self.dims = tuple(shape)
        self.dtype = dtype
        self.device = dev
        return self

    def __reduce__(self):
        return PagedCache, tuple(self)

    def _c(self):
        return _pages([t.data_ptr() for t in self], self.dims, len(self) > 2)

    k = property(lambda self: self[0])
    v = property(lambda self: self[1])
    k_scale = property(lambda self: self[2] if len(self) > 2 else None)
    v_scale = property(lambda self: self[3] if len(self) > 2 else None)


def paged_cache(n_pages, H_kv, page, D, dtype=None, device="cuda"):
    """A zeroed pool of ``n_pages`` pages of ``page`` slots (16, 32, 64 or 128),
    in bfloat16 or, with ``dtype=torch.float8_e4m3fn``, 8 bits."""
    torch = _T or _import_torch()
    if D not in (64, 128) or page not in (16, 32, 64, 128) or n_pages <= 0 or H_kv <= 0:
        raise ValueError("D must be 64 or 128, page 16, 32, 64 or 128, n_pages and H_kv positive")
    dtype = torch.bfloat16 if dtype is None else dtype
    shape = (n_pages, H_kv, page, D)
    parts = [torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)]
    if dtype == torch.float8_e4m3fn:
        parts += [torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2)]
    return PagedCache(*parts)


def _paged_args(cache, table, names, tensors, ints, dev_status):
    """The checks that the paged calls share: ``table`` int32 [B, width], named
    int32 tensors of n elements, and every tensor contiguous on the cache's
    device. Returns the table's width."""
    i32 = _T.int32
    if table.dim() != 2 or table.dtype != i32:
        raise ValueError("table must be int32 [B, width]")
    for t, name, n in ints:
        if t is not None and (t.dtype != i32 or t.shape != (n,)):
            _like(t, name, (n,), i32)
    if dev_status is not None:
        _int_buffer(dev_status, "dev_status", 1)
    _with_cache(cache, tensors, names)
    return table.shape[1]


_APPEND = ("table", "k", "v", "start", "n_new", "dev_status")


def paged_append(cache, table, k, v, start, n_new=None, dev_status=None, stream=None):
    """Writes k, v [B, T, H_kv, D] (bf16 or float32) to slots start[b],
    start[b] + 1, ... of the sequences whose pages ``table`` int32 [B, width]
    names; with ``n_new`` int32 [B] only the first n_new[b] tokens of a padded
    batch. start: int32 [B]. All CUDA tensors."""
    lib = _lib or load()
    _, H_kv, _, D = cache.dims
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4 or shape[2] != H_kv or shape[3] != D:
        raise ValueError(f"k must be [B, T, {H_kv}, {D}]")
    if v.shape != shape or v.dtype != dtype:
        _like(v, "v", shape, dtype)
    B, T = shape[0], shape[1]
    code = _dtype_code(dtype)
    if table.shape[0] != B:
        raise ValueError(f"table must be int32 [{B}, width]")
    width = _paged_args(cache, table, _APPEND, (table, k, v, start, n_new, dev_status),
                        ((start, "start", B), (n_new, "n_new", B)), dev_status)
    st = lib.paged_append(cache._c(), table.data_ptr(), width, k.data_ptr(), v.data_ptr(),
                          start.data_ptr(), _ptr(n_new), B, T, code, _ptr(dev_status),
                          _stream(stream))
    if st:
        _check(st, "paged_append")


_APPEND_VARLEN = ("table", "k", "v", "cu_seqlens", "start", "dev_status")


def paged_append_varlen(cache, table, k, v, cu_seqlens, start, dev_status=None, stream=None):
    """``paged_append`` of packed tokens k, v [total, H_kv, D]: sequence b's are
    rows [cu_seqlens[b], cu_seqlens[b + 1]) (int32 [B + 1], CUDA)."""
    lib = _lib or load()
    _, H_kv, _, D = cache.dims
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or shape[1] != H_kv or shape[2] != D:
        raise ValueError(f"k must be [total, {H_kv}, {D}]")
    if v.shape != shape or v.dtype != dtype:
        _like(v, "v", shape, dtype)
    B = table.shape[0]
    code = _dtype_code(dtype)
    width = _paged_args(cache, table, _APPEND_VARLEN, (table, k, v, cu_seqlens, start, dev_status),
                        ((start, "start", B), (cu_seqlens, "cu_seqlens", B + 1)), dev_status)
    st = lib.paged_append_varlen(cache._c(), table.data_ptr(), width, k.data_ptr(), v.data_ptr(),
                                 start.data_ptr(), cu_seqlens.data_ptr(), B, shape[0], code,
                                 _ptr(dev_status), _stream(stream))
    if st:
        _check(st, "paged_append_varlen")


_READ = ("table", "k", "v", "start", "dev_status")


def paged_read(cache, table, start, T, dtype=None, k=None, v=None, dev_status=None, stream=None):
    """The values (k, v) [B, T, H_kv, D] of slots start[b] ... start[b] + T - 1
    (start None: from slot 0), bf16 unless ``dtype`` or a given k or v says
    float32; zeros where ``table`` int32 [B, width] names no page."""
    torch = _T or _import_torch()
    lib = _lib or load()
    _, H_kv, _, D = cache.dims
    if dtype is None:
        given = k if k is not None else v
        dtype = torch.bfloat16 if given is None else given.dtype
    code = _dtype_code(dtype)
    T = int(T)
    if T <= 0:
        raise ValueError("T must be positive")
    B = table.shape[0]
    shape = (B, T, H_kv, D)
    if k is not None:
        _like(k, "k", shape, dtype)
    if v is not None:
        _like(v, "v", shape, dtype)
    width = _paged_args(cache, table, _READ, (table, k, v, start, dev_status),
                        ((start, "start", B),), dev_status)
    if k is None or v is None:
        if stream is None:
            k = torch.empty(shape, dtype=dtype, device=table.device) if k is None else k
            v = torch.empty_like(k) if v is None else v
        else:
            with torch.cuda.stream(stream):
                k = torch.empty(shape, dtype=dtype, device=table.device) if k is None else k
                v = torch.empty_like(k) if v is None else v
    st = lib.paged_read(cache._c(), table.data_ptr(), width, _ptr(start), k.data_ptr(),
                        v.data_ptr(), B, _int32(T), code, _ptr(dev_status), _stream(stream))
    if st:
        _check(st, "paged_read")
    return k, v


# (a function of the sizes alone; asking the library costs as much as a launch)
@functools.lru_cache(maxsize=256)
def _paged_workspace(dims, quant, B, S_q, total, H_q, max_len, window, n_sink, varlen):
    n = ctypes.c_size_t()
    pages = _pages((0,) * (4 if quant else 2), dims, quant)
    _check(load().paged_attn_workspace(pages, B, S_q, total, H_q, max_len, window, n_sink, varlen,
                                       ctypes.byref(n)), "paged_attn_workspace")
    return n.value


def paged_attn_workspace_bytes(cache, B, S_q, H_q, max_len, window=0, n_sink=0, total=None):
    """Bytes of device workspace that ``paged_attn`` needs for these sizes; with
    ``total``, ``paged_attn_varlen`` of B sequences of at most S_q new tokens in
    ``total`` rows."""
    torch = _T or _import_torch()
    sizes = map(_int32, (B, S_q, 0 if total is None else total, H_q, max_len, window, n_sink))
    return _paged_workspace(cache.dims, cache.dtype == torch.float8_e4m3fn, *sizes,
                            int(total is not None))


_ATTN = ("q", "table", "lens", "cu_seqlens", "out", "lse", "workspace", "dev_status")


def _paged_attn(q, cache, table, lens, cu_seqlens, B, S_q, total, max_len, window, n_sink, scale,
                out, lse, workspace, dev_status, stream):
    """Both forms of the attention; ``cu_seqlens`` None: [B, S_q, H_q, D]."""
    torch = _T or _import_torch()
    lib = _lib or load()
    H_q = q.shape[-2]
    packed = cu_seqlens is not None
    lse_shape = (H_q, total) if packed else (B, H_q, S_q)
    code = _dtype_code(q.dtype)
    if out is not None:
        _like(out, "out", q.shape, q.dtype)
    if lse is not None:
        _like(lse, "lse", lse_shape, torch.float32)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    if table.shape[0] != B:
        raise ValueError(f"table must be int32 [{B}, width]")
    width = _paged_args(cache, table, _ATTN,
                        (q, table, lens, cu_seqlens, out, lse, workspace, dev_status),
                        ((lens, "lens", B), (cu_seqlens, "cu_seqlens", B + 1)), dev_status)
    # (lengths are counted in 30 bits, whatever a table is wide)
    max_len = min(width * cache.dims[2], 1 << 30) if max_len is None else _int32(max_len)
    S_q, window, n_sink = _int32(S_q), _int32(window), _int32(n_sink)
    if out is None or lse is None or workspace is None:
        with _on_stream(stream):
            if out is None:
                out = torch.empty_like(q)
            if lse is None:
                lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
            if workspace is None:
                need = _paged_workspace(cache.dims, len(cache) > 2, B, S_q, total, H_q, max_len,
                                        window, n_sink, packed)
                if need:
                    workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    if packed:
        st = lib.paged_attn_varlen(q.data_ptr(), cache._c(), table.data_ptr(), width,
                                   lens.data_ptr(), cu_seqlens.data_ptr(), out.data_ptr(),
                                   lse.data_ptr(), B, total, S_q, H_q, max_len, window, n_sink, sc,
                                   code, ws, ws_bytes, _ptr(dev_status), _stream(stream))
    else:
        st = lib.paged_attn(q.data_ptr(), cache._c(), table.data_ptr(), width, lens.data_ptr(),
                            out.data_ptr(), lse.data_ptr(), B, S_q, H_q, max_len, window, n_sink,
                            sc, code, ws, ws_bytes, _ptr(dev_status), _stream(stream))
    if st:
        _check(st, "paged_attn_varlen" if packed else "paged_attn")
    return out, lse


def paged_attn(q, cache, table, lens, max_len=None, window=0, n_sink=0, scale=None, out=None,
               lse=None, workspace=None, dev_status=None, stream=None):
    """Attention of new tokens q [B, S_q, H_q, D] (bf16) over the slots that
    ``table`` int32 [B, width] finds in the pages.

    ``lens`` int32 [B] (CUDA) counts the slots in use, the S_q new tokens'
    included; ``max_len`` (default: all that the table is wide) bounds it and
    sizes the launch. ``window`` > 0 limits every query to its last ``window``
    slots and the first ``n_sink``. Returns (out [B, S_q, H_q, D], lse
    [B, H_q, S_q]). A ``workspace`` (uint8, ``paged_attn_workspace_bytes``) is
    allocated here when not given; calls that may overlap need their own.
    """
    shape = q.shape
    if len(shape) != 4 or shape[3] != cache.dims[3]:
        raise ValueError("q must be [B, S_q, H_q, D] matching the cache")
    B, S_q = shape[0], shape[1]
    return _paged_attn(q, cache, table, lens, None, B, S_q, B * S_q, max_len, window, n_sink, scale,
                       out, lse, workspace, dev_status, stream)


def paged_attn_varlen(q, cache, table, lens, cu_seqlens, max_seqlen, max_len=None, window=0,
                      n_sink=0, scale=None, out=None, lse=None, workspace=None, dev_status=None,
                      stream=None):
    """``paged_attn`` of packed tokens q [total, H_q, D]: sequence b's new ones,
    at most ``max_seqlen``, are rows [cu_seqlens[b], cu_seqlens[b + 1]) (int32
    [B + 1], CUDA): pieces of prompts behind what is cached, and single tokens.
    Returns (out [total, H_q, D], lse [H_q, total])."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.dims[3]:
        raise ValueError("q must be [total, H_q, D] matching the cache")
    return _paged_attn(q, cache, table, lens, cu_seqlens, table.shape[0], max_seqlen, shape[0],
                       max_len, window, n_sink, scale, out, lse, workspace, dev_status, stream)


def expiry_test(q, k, v, out, lse, dev_status, stream=None):
    """Launch the kernel with one load withheld (see ring_attn_expiry_test)."""
    lib = load()
    _int_buffer(dev_status, "dev_status", 1)
    _on_device(((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"),
                (dev_status, "dev_status")))
    S = q.shape[1]
    st = lib.ring_attn_expiry_test(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), S,
                                   _ptr(dev_status), _stream(stream))
    _check(st, "ring_attn_expiry_test")

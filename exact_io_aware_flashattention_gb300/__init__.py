"""Thin Python binding of libfa_gb300.so (exact IO-aware attention on GB300).

The names ``fa_fwd``, ``fa_fwd_ex``, ``fa_fwd_ex_workspace_bytes``,
``fa_fwd_ex_default_splits``, ``fa_bwd``, ``fa_bwd_ex``, ``fa_bwd_preprocess``,
``fa_bwd_dkdv``, ``fa_bwd_dq_convert``, ``fa_bwd_workspace_bytes``, ``fa_strerror``,
``fa_last_device_status``, ``fa_selftest_wait_timeout``,
``fa_selftest_drain_timeout``, ``fa_bwd_noalloc``, ``fa_rope``,
``fa_paged_append``, ``fa_paged_decode``, ``fa_paged_decode_workspace_bytes``,
``fa_paged_evict``, ``fa_qk_norm_rope``, ``fa_qk_norm_rope_bwd``,
``fa_qk_norm_rope_bwd_workspace_bytes``, ``fa_paged4_append``, ``fa_paged4_read``,
``fa_paged4_decode``, ``fa_paged4_decode_workspace_bytes``,
``fa_last_cuda_error`` and ``fa_version`` are the C entry points of ``include/fa.h`` with the same arguments (pointers as
Python ints, stream as an int handle); they return the integer status.

``forward``/``backward`` marshal torch CUDA tensors into those calls: they
check dtype, shape, contiguity and device, allocate outputs with torch, pass
``data_ptr()`` and the current stream, and raise ``FAError`` on a non-zero
status.  ``rope``, ``rope_backward``, ``paged_append``, ``paged_decode`` and
``paged_evict`` do the same for rotary positions and the paged key / value
cache; ``qk_norm_rope``, ``qk_norm_rope_backward``, ``paged4_append``,
``paged4_read`` and ``paged4_decode`` for the norms of queries and keys and the
cache held in 4 bits.  Every step of the computation runs in the library's kernels; there
is no fallback of any kind.  If the library has not been built the first call
raises ``FAError``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import re
import struct

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "_lib", "libfa_gb300.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "fa.h")

FA_OK = 0
FA_ERR_NULL_PTR = 1
FA_ERR_BAD_SHAPE = 2
FA_ERR_UNSUPPORTED_HEADDIM = 3
FA_ERR_MISALIGNED = 4
FA_ERR_WORKSPACE_TOO_SMALL = 5
FA_ERR_UNSUPPORTED_DEVICE = 6
FA_ERR_LAUNCH = 7
FA_ERR_DEVICE_TIMEOUT = 8
FA_ERR_CUDA = 9
FA_ERR_BAD_ARGUMENT = 10
FA_ERR_ALIASING = 11
FA_ERR_SCRATCH_LIMIT = 12
FA_ERR_DEVICE_DRAIN = 13
FA_ERR_BAD_INDEX = 14
FA_BF16 = 0
FA_FP16 = 1
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class FAError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: status {status} ({_strerror_safe(status)})" if what else
                         f"status {status} ({_strerror_safe(status)})")


_lib = None

_p = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong


class fa_rotary(ctypes.Structure):
    _fields_ = [("positions", _p), ("axis_stride", _ll), ("batch_stride", _ll), ("inv_freq", _p), ("axes", _p),
                ("n_axes", _i), ("rot", _i), ("interleaved", _i)]


class fa_paged_kv(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("page_stride", _ll), ("head_stride", _ll), ("slot_stride", _ll),
                ("num_pages", _i), ("page_size", _i), ("Hkv", _i), ("d", _i), ("dtype", _i)]


class fa_page_table(ctypes.Structure):
    _fields_ = [("pages", _p), ("stride", _ll), ("max_pages", _i)]


class fa_qk_norm(ctypes.Structure):
    _fields_ = [("q_weight", _p), ("k_weight", _p), ("weights_fp32", _i), ("eps", _f)]


class fa_paged4_kv(ctypes.Structure):
    _fields_ = [("data", _p), ("page_stride", _ll), ("head_stride", _ll), ("num_pages", _i), ("page_size", _i),
                ("Hkv", _i), ("d", _i), ("dtype", _i)]


_SIGNATURES = {
    "fa_fwd": ([_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p], _i),
    "fa_fwd_ex": ([_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_fwd_ex_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i], _sz),
    "fa_fwd_ex_default_splits": ([_i, _i, _i, _i, _i, _i, _i, _i], _i),
    "fa_bwd_ex": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_bwd_workspace_bytes": ([_i, _i, _i, _i, _i], _sz),
    "fa_bwd": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_bwd_preprocess": ([_p, _p, _p, _i, _i, _i, _i, _i, _p, _sz, _p], _i),
    "fa_bwd_dkdv": ([_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_bwd_dq_convert": ([_p, _i, _i, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_strerror": ([_i], ctypes.c_char_p),
    "fa_last_device_status": ([_p, ctypes.POINTER(ctypes.c_int)], _i),
    "fa_selftest_wait_timeout": ([ctypes.c_ulonglong, _p], _i),
    "fa_selftest_drain_timeout": ([ctypes.c_ulonglong, _p], _i),
    "fa_version": ([], _i),
    "fa_last_cuda_error": ([], ctypes.c_char_p),
    "fa_bwd_noalloc": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p], _i),
    "fa_rope": ([_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _i, _p], _i),
    "fa_paged_append": ([_p, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _i, _p, _p, _p], _i),
    "fa_paged_decode": ([_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_paged_decode_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i], _sz),
    "fa_paged_evict": ([_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _p], _i),
    "fa_qk_norm_rope": ([_p] * 8 + [_i] * 6 + [_p, _p, _p], _i),
    "fa_qk_norm_rope_bwd": ([_p] * 14 + [_i] * 6 + [_p, _p, _p, _sz, _p], _i),
    "fa_qk_norm_rope_bwd_workspace_bytes": ([_i], _sz),
    "fa_paged4_append": ([_p, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _i, _p, _p, _p], _i),
    "fa_paged4_read": ([_p, _p, _p, _p, _p, _p, _p, _i, _i, _p], _i),
    "fa_paged4_decode": ([_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _f, _p, _sz, _p], _i),
    "fa_paged4_decode_workspace_bytes": ([_i, _i, _i, _i], _sz),
}


def load_library(path: str | None = None):
    """Load (once) and return the ctypes handle; raises FAError if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FAError(FA_ERR_LAUNCH, f"CUDA library not built at {p} (run __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def header_functions(path: str = HEADER_PATH) -> list[str]:
    """Names of the functions include/fa.h declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_]\w*\s*\**\s*(fa_\w+)\s*\(", text, flags=re.M)))


def _strerror_safe(status: int) -> str:
    try:
        return load_library().fa_strerror(status).decode()
    except Exception:
        return "library not loaded"


# ---------------------------------------------------------------------------
# Raw entry points (same names and arguments as the C ABI).
# ---------------------------------------------------------------------------

def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream):
    return load_library().fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, int(causal), float(scale), stream)


def fa_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, window, num_splits, scale, workspace,
              workspace_bytes, stream):
    return load_library().fa_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, int(causal), int(window),
                                     int(num_splits), float(scale), workspace, workspace_bytes, stream)


def fa_fwd_ex_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits):
    return load_library().fa_fwd_ex_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits)


def fa_fwd_ex_default_splits(B, Hq, Hkv, Nq, Nk, d, causal, window):
    return load_library().fa_fwd_ex_default_splits(B, Hq, Hkv, Nq, Nk, d, int(causal), int(window))


def fa_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, window, deterministic, scale, workspace,
              workspace_bytes, stream):
    return load_library().fa_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, N, d, int(causal), int(window),
                                    int(deterministic), float(scale), workspace, workspace_bytes, stream)


def fa_bwd_workspace_bytes(B, Hq, Hkv, N, d):
    return load_library().fa_bwd_workspace_bytes(B, Hq, Hkv, N, d)


def fa_bwd(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes, stream):
    return load_library().fa_bwd(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, N, d, int(causal), float(scale),
                                 workspace, workspace_bytes, stream)


def fa_bwd_preprocess(o, do, lse, B, Hq, Hkv, N, d, workspace, workspace_bytes, stream):
    return load_library().fa_bwd_preprocess(o, do, lse, B, Hq, Hkv, N, d, workspace, workspace_bytes, stream)


def fa_bwd_dkdv(q, k, v, do, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes, stream):
    return load_library().fa_bwd_dkdv(q, k, v, do, dk, dv, B, Hq, Hkv, N, d, int(causal), float(scale),
                                      workspace, workspace_bytes, stream)


def fa_bwd_dq_convert(dq, B, Hq, Hkv, N, d, scale, workspace, workspace_bytes, stream):
    return load_library().fa_bwd_dq_convert(dq, B, Hq, Hkv, N, d, float(scale), workspace, workspace_bytes, stream)


def fa_strerror(status):
    return load_library().fa_strerror(status).decode()


def fa_last_device_status(stream=None):
    """Return (status, (block, site, thread))."""
    detail = (ctypes.c_int * 3)()
    s = load_library().fa_last_device_status(stream, detail)
    return s, tuple(detail)


def fa_selftest_wait_timeout(timeout_ns, stream=None):
    return load_library().fa_selftest_wait_timeout(int(timeout_ns), stream)


def fa_selftest_drain_timeout(timeout_ns, stream=None):
    return load_library().fa_selftest_drain_timeout(int(timeout_ns), stream)


def fa_version():
    return load_library().fa_version()


def fa_last_cuda_error():
    return load_library().fa_last_cuda_error().decode()


def fa_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, stream):
    """fa_bwd without a workspace argument: the scratch is a fixed buffer inside
    the library (for callers that cannot allocate device memory)."""
    return load_library().fa_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, B, Hq, Hkv, N, d, int(causal),
                                         float(scale), stream)


def _ref(s):
    return ctypes.byref(s) if isinstance(s, ctypes.Structure) else s


def fa_rope(q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides, B, Hq, Hk, N, d, dtype, rotary,
            inverse, stream):
    return load_library().fa_rope(q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides, B, Hq, Hk, N,
                                  d, dtype, _ref(rotary), int(inverse), stream)


def fa_paged_append(kv, table, seq_lens, cu_seqlens, B, T, k, k_strides, v, v_strides, q, q_strides, q_out,
                    q_out_strides, Hq, rotary, scores, stream):
    return load_library().fa_paged_append(_ref(kv), _ref(table), seq_lens, cu_seqlens, B, T, k, k_strides, v, v_strides,
                                          q, q_strides, q_out, q_out_strides, Hq, _ref(rotary), scores, stream)


def fa_paged_decode(q, q_strides, kv, table, seq_lens, o, lse, scores, B, Hq, window, scale, workspace,
                    workspace_bytes, stream):
    return load_library().fa_paged_decode(q, q_strides, _ref(kv), _ref(table), seq_lens, o, lse, scores, B, Hq,
                                          int(window), float(scale), workspace, workspace_bytes, stream)


def fa_paged_decode_workspace_bytes(B, Hq, Hkv, d, page_size, max_pages, with_scores):
    return load_library().fa_paged_decode_workspace_bytes(B, Hq, Hkv, d, page_size, max_pages, int(with_scores))


def fa_paged_evict(kv, scores, table, seq_lens, dst, new_lens, kept, B, budget, recent, sinks, stream):
    return load_library().fa_paged_evict(_ref(kv), scores, _ref(table), seq_lens, _ref(dst), new_lens, kept, B,
                                         int(budget), int(recent), int(sinks), stream)


def fa_qk_norm_rope(q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides, B, Hq, Hk, N, d, dtype, norm,
                    rotary, stream):
    return load_library().fa_qk_norm_rope(q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides, B, Hq,
                                          Hk, N, d, dtype, _ref(norm), _ref(rotary), stream)


def fa_qk_norm_rope_bwd(dq_out, dq_out_strides, q, q_strides, dq, dq_strides, dk_out, dk_out_strides, k, k_strides, dk,
                        dk_strides, dq_weight, dk_weight, B, Hq, Hk, N, d, dtype, norm, rotary, workspace,
                        workspace_bytes, stream):
    return load_library().fa_qk_norm_rope_bwd(dq_out, dq_out_strides, q, q_strides, dq, dq_strides, dk_out,
                                              dk_out_strides, k, k_strides, dk, dk_strides, dq_weight, dk_weight, B, Hq,
                                              Hk, N, d, dtype, _ref(norm), _ref(rotary), workspace, workspace_bytes,
                                              stream)


def fa_qk_norm_rope_bwd_workspace_bytes(d):
    return load_library().fa_qk_norm_rope_bwd_workspace_bytes(d)


def fa_paged4_append(kv, table, seq_lens, cu_seqlens, B, T, k, k_strides, v, v_strides, q, q_strides, q_out,
                     q_out_strides, Hq, norm, rotary, stream):
    return load_library().fa_paged4_append(_ref(kv), _ref(table), seq_lens, cu_seqlens, B, T, k, k_strides, v, v_strides,
                                           q, q_strides, q_out, q_out_strides, Hq, _ref(norm), _ref(rotary), stream)


def fa_paged4_read(kv, table, seq_lens, k, k_strides, v, v_strides, B, N, stream):
    return load_library().fa_paged4_read(_ref(kv), _ref(table), seq_lens, k, k_strides, v, v_strides, B, N, stream)


def fa_paged4_decode(q, q_strides, kv, table, seq_lens, o, lse, B, Hq, window, scale, workspace, workspace_bytes, stream):
    return load_library().fa_paged4_decode(q, q_strides, _ref(kv), _ref(table), seq_lens, o, lse, B, Hq, int(window),
                                           float(scale), workspace, workspace_bytes, stream)


def fa_paged4_decode_workspace_bytes(B, Hq, Hkv, d):
    return load_library().fa_paged4_decode_workspace_bytes(B, Hq, Hkv, d)


# ---------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------

def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(t, name, shape, dtype):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raise(status, what):
    if status != FA_OK:
        if status in (FA_ERR_LAUNCH, FA_ERR_CUDA):
            what = f"{what} [{fa_last_cuda_error()}]"
        raise FAError(status, what)


def forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, stream=None):
    """O, LSE = exact attention of bf16 [B,Hq,N,d] q and [B,Hkv,N,d] k, v."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    _check(q, "q", (B, Hq, N, d), torch.bfloat16)
    _check(k, "k", (B, Hkv, N, d), torch.bfloat16)
    _check(v, "v", (B, Hkv, N, d), torch.bfloat16)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    _check(out, "out", (B, Hq, N, d), torch.bfloat16)
    _check(lse, "lse", (B, Hq, N), torch.float32)
    _raise(fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                  B, Hq, Hkv, N, d, causal, scale, _stream_handle(stream)), "fa_fwd")
    return out, lse


def forward_ex(q, k, v, causal: bool = False, scale: float | None = None, window: int = 0, num_splits: int = 1,
               out=None, lse=None, workspace=None, stream=None):
    """O, LSE of bf16 q [B,Hq,Nq,d] against k, v [B,Hkv,Nk,d] (queries at the last
    Nq positions), with an optional sliding window and key splits; see fa_fwd_ex.
    ``num_splits=0`` takes fa_fwd_ex_default_splits."""
    import torch
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(q, "q", (B, Hq, Nq, d), torch.bfloat16)
    _check(k, "k", (B, Hkv, Nk, d), torch.bfloat16)
    _check(v, "v", (B, Hkv, Nk, d), torch.bfloat16)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if num_splits == 0:
        num_splits = fa_fwd_ex_default_splits(B, Hq, Hkv, Nq, Nk, d, causal, window)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    _check(out, "out", (B, Hq, Nq, d), torch.bfloat16)
    _check(lse, "lse", (B, Hq, Nq), torch.float32)
    nbytes = fa_fwd_ex_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    wp = workspace.data_ptr() if workspace is not None else None
    wn = workspace.numel() if workspace is not None else 0
    _raise(fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Nq, Nk,
                     d, causal, window, num_splits, scale, wp, wn, _stream_handle(stream)), "fa_fwd_ex")
    return out, lse


def workspace_for(B, Hq, Hkv, N, d, device):
    import torch
    nbytes = fa_bwd_workspace_bytes(B, Hq, Hkv, N, d)
    if nbytes == 0:
        raise FAError(FA_ERR_BAD_SHAPE, "fa_bwd_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def backward(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, workspace=None,
             dq=None, dk=None, dv=None, stream=None, window: int = 0, deterministic: bool = False):
    """dQ, dK, dV of sum(dO * O), recomputing P from the forward's LSE."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    for t, name, hh in ((q, "q", Hq), (k, "k", Hkv), (v, "v", Hkv), (o, "o", Hq), (do, "do", Hq)):
        _check(t, name, (B, hh, N, d), torch.bfloat16)
    _check(lse, "lse", (B, Hq, N), torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = workspace_for(B, Hq, Hkv, N, d, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _raise(fa_bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, N, d, causal, window, deterministic, scale,
                     workspace.data_ptr(), workspace.numel(), _stream_handle(stream)), "fa_bwd_ex")
    return dq, dk, dv


def check_device_status(stream=None):
    """Raise FAError if a kernel of this library recorded a device-side error."""
    s, detail = fa_last_device_status(_stream_handle(stream))
    if s != FA_OK:
        raise FAError(s, f"device status (block, site, thread) = {detail}")


# ---------------------------------------------------------------------------
# Rotary positions and the paged key / value cache
#
# A decoding step makes these calls for every layer on tensors of a few KB, so
# their time is the binding's.  The public functions first offer a call to the
# native marshalling (csrc/fa_torch.cpp), which takes what is in order, on the
# current device and stream; what it does not take, because something is wrong
# or elsewhere, or because it has not been built, goes through the functions
# below, which say what is wrong.  There the checks of a valid argument are one
# expression, structs and stride arrays packed bytes, the stream a raw handle.
# ---------------------------------------------------------------------------

class _NotBuilt:
    """Stands for the native marshalling where there is none: takes no call."""

    @staticmethod
    def _none(*args):
        return None
    rope = paged_append = paged_decode = paged_evict = _none
    qk_norm_rope = qk_norm_rope_backward = paged4_append = paged4_read = paged4_decode = _none


_native = None


def _load_native():
    """The native marshalling, bound to the library's entry points."""
    global _native
    lib = load_library()
    path = os.path.join(os.path.dirname(LIB_PATH), "fa_torch.so")
    _native = _NotBuilt
    if os.path.exists(path):
        import importlib.util
        import torch  # noqa: F401  (its libraries, which the module needs, are then loaded)
        from . import _build
        try:
            spec = importlib.util.spec_from_file_location("fa_torch", path)
            m = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(m)
            if getattr(m, "key", None) == _build.native_key():
                m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                    lib.fa_rope, lib.fa_paged_append, lib.fa_paged_decode, lib.fa_paged_decode_workspace_bytes,
                    lib.fa_paged_evict, lib.fa_qk_norm_rope, lib.fa_qk_norm_rope_bwd,
                    lib.fa_qk_norm_rope_bwd_workspace_bytes, lib.fa_paged4_append, lib.fa_paged4_read,
                    lib.fa_paged4_decode, lib.fa_paged4_decode_workspace_bytes)))
                _native = m
        except ImportError:          # built against another torch
            pass
    return _native


def native_marshalling() -> bool:
    """Whether calls are marshalled natively (see build's fa_torch.txt if not)."""
    return (_native or _load_native()) is not _NotBuilt


def _answer(r, what):
    """The native marshalling's answer: outputs, or a status to raise."""
    if type(r) is int:
        _raise(r, what)
    return r

_pack_rotary = struct.Struct("@PqqPPiii4x").pack          # fa_rotary
_pack_kv = struct.Struct("@PPqqqiiiii4x").pack            # fa_paged_kv
_pack_table = struct.Struct("@Pqi4x").pack                # fa_page_table
_pack2 = struct.Struct("@qq").pack
_pack3 = struct.Struct("@qqq").pack


def _check_view(t, name, shape, dtype, dev):
    """Address of a tensor of this shape on CUDA device ``dev``, contiguous in its last dimension."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.stride()[-1] == 1:
            return t.data_ptr()
    except (AttributeError, IndexError):
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr()


def _check_dense(t, name, shape, dtype, dev):
    """Address of a contiguous tensor."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check_view(t, name, shape, dtype, dev)
    raise ValueError(f"{name} must be contiguous")


_torch = None           # the torch module, and its queries of the current device and stream,
_current_device = None  # once the first call has imported it
_current_stream = None


def _load_torch():
    global _torch, _current_device, _current_stream
    import torch
    _torch, _current_device, _current_stream = torch, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _first(t, name, dims, what):
    """(shape, CUDA device index, dtype code, dtype) of a call's first tensor."""
    if _torch is None:
        _load_torch()
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape, dt = t.shape, t.dtype
    if len(shape) != dims:
        raise ValueError(f"{name} must be a {what} tensor, got shape {tuple(shape)}")
    if dt is _torch.bfloat16:
        code = FA_BF16
    elif dt is _torch.float16:
        code = FA_FP16
    else:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {dt}")
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    return shape, dev, code, dt


def _raw_stream(dev, stream):
    """Handle of device ``dev``'s current stream if that device is current and no
    other stream is asked for, else None: the call is then made again inside
    ``_on``, so that what it allocates belongs to the stream it runs on (the
    caching allocator would else hand a workspace on to another stream while the
    kernels still use it)."""
    return _current_stream(dev) if stream is None and dev == _current_device() else None


@contextlib.contextmanager
def _on(dev, stream):
    """Device ``dev`` and ``stream`` (None: the device's current stream) made current."""
    import torch
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream of {stream.device}, tensors on cuda:{dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield


def _rotary(positions, inv_freq, axes, interleaved, d, lead, dev):
    """fa_rotary of positions [n_axes, *lead] int32, inv_freq [rot/2] float64, axes [rot/2] int32."""
    try:
        n_axes, n, st = positions.shape[0], inv_freq.shape[0], positions.stride()
    except (AttributeError, IndexError):
        raise ValueError("rotary positions need positions, inv_freq and axes as tensors") from None
    pos = _check_view(positions, "positions", (n_axes, *lead), _torch.int32, dev)
    if n < 1 or 2 * n > d:
        raise ValueError(f"inv_freq has {n} frequencies, expected 1 to {d // 2}")
    w = _check_dense(inv_freq, "inv_freq", (n,), _torch.float64, dev)
    ax = _check_dense(axes, "axes", (n,), _torch.int32, dev)
    return _pack_rotary(pos, st[0], st[1] if len(lead) == 2 else 0, w, ax, n_axes, 2 * n, 1 if interleaved else 0)


def rope_frequencies(sections, base: float = 10000.0, device="cuda"):
    """inv_freq [r] float64 and axes [r] int32 for ``rope``: the r = sum(sections)
    pairs have the frequencies base^(-i/r) and are dealt to the axes in runs of
    ``sections`` pairs, e.g. (64,) for text at d = 128 or (16, 24, 24) for time,
    height and width.  Any other two arrays of these types do as well."""
    import torch
    r = sum(sections)
    if r < 1 or min(sections) < 0:
        raise ValueError("sections must be non-negative with a positive sum")
    inv = float(base) ** (-torch.arange(r, dtype=torch.float64) / r)
    axes = torch.repeat_interleave(torch.arange(len(sections), dtype=torch.int32), torch.tensor(sections))
    return inv.to(device), axes.to(device)


def _rope(q, k, positions, inv_freq, axes, interleaved, inverse, q_out, k_out, stream):
    (B, Hq, N, d), dev, code, dt = _first(q, "q", 4, "[B, Hq, N, d]")
    qp = _check_view(q, "q", q.shape, dt, dev)
    Hk, kp, ks = 0, None, None
    if k is not None:
        Hk = k.shape[1] if isinstance(k, _torch.Tensor) and k.dim() == 4 else 0
        kp = _check_view(k, "k", (B, Hk, N, d), dt, dev)
        ks = _pack3(*k.stride()[:3])
    elif k_out is not None:
        raise ValueError("k_out without k")
    rot = _rotary(positions, inv_freq, axes, interleaved, d, (B, N), dev)
    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _rope(q, k, positions, inv_freq, axes, interleaved, inverse, q_out, k_out, None)
    if q_out is None:
        q_out = _torch.empty((B, Hq, N, d), dtype=dt, device=q.device)
        op = q_out.data_ptr()
    else:
        op = _check_view(q_out, "q_out", (B, Hq, N, d), dt, dev)
    okp, oks = None, None
    if k is not None:
        if k_out is None:
            k_out = _torch.empty((B, Hk, N, d), dtype=dt, device=q.device)
            okp = k_out.data_ptr()
        else:
            okp = _check_view(k_out, "k_out", (B, Hk, N, d), dt, dev)
        oks = _pack3(*k_out.stride()[:3])
    status = fa_rope(qp, _pack3(*q.stride()[:3]), op, _pack3(*q_out.stride()[:3]), kp, ks, okp, oks, B, Hq, Hk, N, d, code,
                     rot, inverse, handle)
    if status:
        _raise(status, "fa_rope")
    return q_out if k is None else (q_out, k_out)


def rope(q, k, positions, inv_freq, axes, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """q [B,Hq,N,d] and k [B,Hk,N,d] (bf16 or fp16, any strides over B, H, N; k may
    be None) with their first 2*len(inv_freq) elements turned: pair i by
    positions[axes[i], b, n] * inv_freq[i] radians; see fa_rope.  positions is
    int32 [n_axes, B, N] (expand over B to share them); inv_freq (float64) and
    axes (int32) come from ``rope_frequencies`` or the caller.  Outputs may be the
    inputs themselves.  Returns (q_out, k_out), or q_out without k."""
    if stream is None:
        r = (_native or _load_native()).rope(q, k, positions, inv_freq, axes, interleaved, False, q_out, k_out)
        if r is not None:
            return _answer(r, "fa_rope")
    return _rope(q, k, positions, inv_freq, axes, interleaved, False, q_out, k_out, stream)


def rope_backward(dq, dk, positions, inv_freq, axes, interleaved: bool = False, dq_out=None, dk_out=None, stream=None):
    """Gradients of ``rope``'s inputs from those of its outputs: the opposite turn."""
    if stream is None:
        r = (_native or _load_native()).rope(dq, dk, positions, inv_freq, axes, interleaved, True, dq_out, dk_out)
        if r is not None:
            return _answer(r, "fa_rope")
    return _rope(dq, dk, positions, inv_freq, axes, interleaved, True, dq_out, dk_out, stream)


def _paged(k_cache, v_cache, block_table, seq_lens):
    """Checked cache tensors: (shape, device index, dtype, fa_paged_kv, fa_page_table, B, seq_lens address)."""
    shape, dev, code, dt = _first(k_cache, "k_cache", 4, "[pages, Hkv, page_size, d]")
    kp = _check_view(k_cache, "k_cache", shape, dt, dev)
    vp = _check_view(v_cache, "v_cache", shape, dt, dev)
    st = k_cache.stride()
    if v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must have the same strides")
    P, Hkv, ps, d = shape
    table, B = _table(block_table, "block_table", dev)
    return (shape, dev, dt, _pack_kv(kp, vp, st[0], st[1], st[2], P, ps, Hkv, d, code), table, B,
            _check_dense(seq_lens, "seq_lens", (B,), _torch.int32, dev))


def _table(t, name, dev):
    shape = t.shape if isinstance(t, _torch.Tensor) and t.dim() == 2 else ("B", "pages")
    return _pack_table(_check_view(t, name, shape, _torch.int32, dev), t.stride()[0], shape[1]), shape[0]


def paged_append(k_cache, v_cache, block_table, seq_lens, k, v, cu_seqlens=None, q=None, positions=None, inv_freq=None,
                 axes=None, interleaved: bool = False, scores=None, q_out=None, stream=None):
    """Store new tokens' k, v [T,Hkv,d] in the paged cache [pages,Hkv,page_size,d].

    ``seq_lens`` [B] int32 includes the new tokens.  Without ``cu_seqlens`` token
    b is the last of sequence b (length 0: padding, skipped); with it ([B+1]
    int32) tokens cu[b]..cu[b+1]-1 are sequence b's last ones and tokens from
    cu[B] on are padding.  With ``positions`` [n_axes,T], ``inv_freq`` and
    ``axes`` k is stored turned, and q [T,Hq,d], if given, is returned turned
    (into ``q_out``, which may be q); rows of padding tokens are not written.
    ``scores`` [pages,Hkv,page_size] fp32 gets 0 for the new tokens.  See
    fa_paged_append."""
    if stream is None:
        r = (_native or _load_native()).paged_append(k_cache, v_cache, block_table, seq_lens, k, v, cu_seqlens, q, positions,
                                                     inv_freq, axes, interleaved, scores, q_out)
        if r is not None:
            return None if r is False else _answer(r, "fa_paged_append")
    return _paged_append(k_cache, v_cache, block_table, seq_lens, k, v, cu_seqlens, q, positions, inv_freq, axes,
                         interleaved, scores, q_out, stream)


def _paged_append(k_cache, v_cache, block_table, seq_lens, k, v, cu_seqlens, q, positions, inv_freq, axes, interleaved,
                  scores, q_out, stream):
    (_, Hkv, _, d), dev, dt, kv, table, B, lens = _paged(k_cache, v_cache, block_table, seq_lens)
    T = k.shape[0] if isinstance(k, _torch.Tensor) and k.dim() == 3 else 0
    kp = _check_view(k, "k", (T, Hkv, d), dt, dev)
    vp = _check_view(v, "v", (T, Hkv, d), dt, dev)
    if cu_seqlens is None:
        cu = None
        if T != B:
            raise ValueError(f"{T} tokens for {B} sequences without cu_seqlens")
    else:
        cu = _check_dense(cu_seqlens, "cu_seqlens", (B + 1,), _torch.int32, dev)
    rot = None
    if positions is not None or inv_freq is not None or axes is not None:
        rot = _rotary(positions, inv_freq, axes, interleaved, d, (T,), dev)
    sp = None if scores is None else _check_dense(scores, "scores", k_cache.shape[:3], _torch.float32, dev)
    qp, qs, Hq = None, None, 0
    if q is not None:
        Hq = q.shape[1] if isinstance(q, _torch.Tensor) and q.dim() == 3 else 0
        qp = _check_view(q, "q", (T, Hq, d), dt, dev)
        qs = _pack2(*q.stride()[:2])
    elif q_out is not None:
        raise ValueError("q_out without q")

    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _paged_append(k_cache, v_cache, block_table, seq_lens, k, v, cu_seqlens, q, positions, inv_freq, axes,
                                 interleaved, scores, q_out, None)
    op, os_ = None, None
    if q is not None:
        if q_out is None:
            q_out = _torch.empty((T, Hq, d), dtype=dt, device=q.device)
            op = q_out.data_ptr()
        else:
            op = _check_view(q_out, "q_out", (T, Hq, d), dt, dev)
        os_ = _pack2(*q_out.stride()[:2])
    if T:
        status = fa_paged_append(kv, table, lens, cu, B, T, kp, _pack2(*k.stride()[:2]), vp, _pack2(*v.stride()[:2]), qp, qs,
                                 op, os_, Hq, rot, sp, handle)
        if status:
            _raise(status, "fa_paged_append")
    return q_out


# A size is a pure function of the shapes; a decoding loop asks for the same one every step.
_decode_ws_bytes = functools.lru_cache(maxsize=256)(
    lambda *shape: fa_paged_decode_workspace_bytes(*shape))


def paged_decode_workspace(B, Hq, k_cache, block_table, with_scores: bool = False):
    """Workspace of paged_decode, for callers that keep one (one for each call that may run at the same time)."""
    import torch
    n = _decode_ws_bytes(B, Hq, k_cache.shape[1], k_cache.shape[3], k_cache.shape[2], block_table.shape[1], bool(with_scores))
    if n == 0:
        raise FAError(FA_ERR_BAD_SHAPE, "fa_paged_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=k_cache.device)


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None, window: int = 0, scores=None,
                 out=None, lse=None, workspace=None, stream=None):
    """O [B,Hq,d], LSE [B,Hq] of one query row per sequence, q [B,Hq,d], against the
    seq_lens[b] keys of the paged cache (the last ``window`` of them if window >
    0).  ``scores`` [pages,Hkv,page_size] fp32, if given, grows at each visible
    key by its softmax weight summed over the group's heads.  See
    fa_paged_decode."""
    if stream is None:
        r = (_native or _load_native()).paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, scores, out,
                                                     lse, workspace)
        if r is not None:
            return _answer(r, "fa_paged_decode")
    return _paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, scores, out, lse, workspace, stream)


def _paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, scores, out, lse, workspace, stream):
    (_, _, _, d), dev, dt, kv, table, B, lens = _paged(k_cache, v_cache, block_table, seq_lens)
    Hq = q.shape[1] if isinstance(q, _torch.Tensor) and q.dim() == 3 else 0
    qp = _check_view(q, "q", (B, Hq, d), dt, dev)
    sp = None if scores is None else _check_dense(scores, "scores", k_cache.shape[:3], _torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)

    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, scores, out, lse, workspace, None)
    device = k_cache.device
    if out is None:
        out = _torch.empty((B, Hq, d), dtype=dt, device=device)
        op = out.data_ptr()
    else:
        op = _check_dense(out, "out", (B, Hq, d), dt, dev)
    if lse is None:
        lse = _torch.empty((B, Hq), dtype=_torch.float32, device=device)
        lp = lse.data_ptr()
    else:
        lp = _check_dense(lse, "lse", (B, Hq), _torch.float32, dev)
    if workspace is None:
        workspace = paged_decode_workspace(B, Hq, k_cache, block_table, scores is not None)
        n, wp = workspace.numel(), workspace.data_ptr()
    else:
        n = workspace.numel()
        wp = _check_dense(workspace, "workspace", (n,), _torch.uint8, dev)
    status = fa_paged_decode(qp, _pack2(*q.stride()[:2]), kv, table, lens, op, lp, sp, B, Hq, window, scale, wp, n, handle)
    if status:
        _raise(status, "fa_paged_decode")
    return out, lse


def paged_evict(k_cache, v_cache, scores, block_table, seq_lens, dst_table, budget: int, recent: int = 0, sinks: int = 0,
                new_lens=None, kept=None, stream=None):
    """Keep min(seq_lens[b], budget) keys of every sequence and kv head: the first
    ``sinks``, the last ``recent``, and those of the rest with the largest
    ``scores``; their K, V and scores are written in order into the pages of
    ``dst_table`` [B, >= ceil(budget/page_size)], which must be other pages than
    those in use.  Returns (new_lens [B], kept [B,Hkv,budget]: the indices kept,
    -1 past the new length).  See fa_paged_evict."""
    if stream is None:
        r = (_native or _load_native()).paged_evict(k_cache, v_cache, scores, block_table, seq_lens, dst_table, budget, recent,
                                                    sinks, new_lens, kept)
        if r is not None:
            return _answer(r, "fa_paged_evict")
    return _paged_evict(k_cache, v_cache, scores, block_table, seq_lens, dst_table, budget, recent, sinks, new_lens, kept,
                        stream)


def _paged_evict(k_cache, v_cache, scores, block_table, seq_lens, dst_table, budget, recent, sinks, new_lens, kept, stream):
    (_, Hkv, _, _), dev, _, kv, table, B, lens = _paged(k_cache, v_cache, block_table, seq_lens)
    sp = _check_dense(scores, "scores", k_cache.shape[:3], _torch.float32, dev)
    dst, rows = _table(dst_table, "dst_table", dev)
    if rows != B:
        raise ValueError(f"dst_table has {rows} rows, expected {B}")
    if budget < 1:
        raise ValueError("budget must be at least 1")

    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _paged_evict(k_cache, v_cache, scores, block_table, seq_lens, dst_table, budget, recent, sinks, new_lens,
                                kept, None)
    if new_lens is None:
        new_lens = _torch.empty((B,), dtype=_torch.int32, device=k_cache.device)
        np_ = new_lens.data_ptr()
    else:
        np_ = _check_dense(new_lens, "new_lens", (B,), _torch.int32, dev)
    if kept is None:
        kept = _torch.empty((B, Hkv, budget), dtype=_torch.int32, device=k_cache.device)
        ip = kept.data_ptr()
    else:
        ip = _check_dense(kept, "kept", (B, Hkv, budget), _torch.int32, dev)
    status = fa_paged_evict(kv, sp, table, lens, dst, np_, ip, B, budget, recent, sinks, handle)
    if status:
        _raise(status, "fa_paged_evict")
    return new_lens, kept


# ---------------------------------------------------------------------------
# Norms of queries and keys, and the cache held in 4 bits
# ---------------------------------------------------------------------------
_pack_norm = struct.Struct("@PPif").pack                  # fa_qk_norm
_pack_kv4 = struct.Struct("@Pqqiiiii4x").pack             # fa_paged4_kv


def _norm(q_weight, k_weight, eps, d, dt, dev):
    """fa_qk_norm of weights [d] (fp32 or the tensors' type, both alike; None: ones)."""
    fp32, ptrs = 0, []
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is None:
            ptrs.append(None)
            continue
        if isinstance(w, _torch.Tensor) and w.dtype is _torch.float32:
            fp32 = 1
        ptrs.append((w, name))
    ptrs = [0 if p is None else _check_dense(p[0], p[1], (d,), _torch.float32 if fp32 else dt, dev) for p in ptrs]
    return _pack_norm(ptrs[0], ptrs[1], fp32, float(eps))


def _maybe_rotary(positions, inv_freq, axes, interleaved, d, lead, dev):
    if positions is None and inv_freq is None and axes is None:
        return None
    return _rotary(positions, inv_freq, axes, interleaved, d, lead, dev)


def _rows_like(t, name, shape, dt, dev):
    """(tensor, address, packed strides) of a given output, or of a new one."""
    if t is None:
        t = _torch.empty(shape, dtype=dt, device=_torch.device("cuda", dev))
        p = t.data_ptr()
    else:
        p = _check_view(t, name, shape, dt, dev)
    return t, p, struct.pack("@%dq" % (len(shape) - 1), *t.stride()[:-1])


def qk_norm_rope(q, k, q_weight, k_weight, positions=None, inv_freq=None, axes=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """``rope`` with the norm of each head's rows in front of it, in one pass: q
    [B,Hq,N,d] and k [B,Hk,N,d] (k may be None) times (mean of squares + eps)^-1/2
    times their weights [d] (fp32 or the tensors' type; None: ones), then turned
    as by ``rope``; without ``positions``, ``inv_freq`` and ``axes`` they are normed
    only.  Outputs may be the inputs themselves.  Returns (q_out, k_out), or q_out
    without k.  See fa_qk_norm_rope."""
    if stream is None:
        r = (_native or _load_native()).qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, q_out, k_out)
        if r is not None:
            return _answer(r, "fa_qk_norm_rope")
    return _qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, q_out, k_out, stream)


def _qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, q_out, k_out, stream):
    (B, Hq, N, d), dev, code, dt = _first(q, "q", 4, "[B, Hq, N, d]")
    qp = _check_view(q, "q", q.shape, dt, dev)
    Hk, kp, ks = 0, None, None
    if k is not None:
        Hk = k.shape[1] if isinstance(k, _torch.Tensor) and k.dim() == 4 else 0
        kp = _check_view(k, "k", (B, Hk, N, d), dt, dev)
        ks = _pack3(*k.stride()[:3])
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out or k_weight without k")
    norm = _norm(q_weight, k_weight, eps, d, dt, dev)
    rot = _maybe_rotary(positions, inv_freq, axes, interleaved, d, (B, N), dev)
    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, q_out, k_out, None)
    q_out, op, os_ = _rows_like(q_out, "q_out", (B, Hq, N, d), dt, dev)
    okp, oks = None, None
    if k is not None:
        k_out, okp, oks = _rows_like(k_out, "k_out", (B, Hk, N, d), dt, dev)
    status = fa_qk_norm_rope(qp, _pack3(*q.stride()[:3]), op, os_, kp, ks, okp, oks, B, Hq, Hk, N, d, code, norm, rot, handle)
    if status:
        _raise(status, "fa_qk_norm_rope")
    return q_out if k is None else (q_out, k_out)


def qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions=None, inv_freq=None, axes=None, eps: float = 1e-6,
                          interleaved: bool = False, dq_out=None, dk_out=None, dq_weight=None, dk_weight=None,
                          workspace=None, stream=None):
    """Gradients of ``qk_norm_rope``'s inputs q and k and of its weights from those
    of its outputs, dq and dk.  Returns (dq, dk, dq_weight, dk_weight), or (dq,
    dq_weight) without k (dk None too); the weights' gradients are fp32 [d], None
    for weights that are None.  ``dq_out`` and ``dk_out`` may be dq and dk
    themselves.  See fa_qk_norm_rope_bwd."""
    if stream is None:
        r = (_native or _load_native()).qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved,
                                                              dq_out, dk_out, dq_weight, dk_weight, workspace)
        if r is not None:
            return _answer(r, "fa_qk_norm_rope_bwd")
    return _qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, dq_out,
                                  dk_out, dq_weight, dk_weight, workspace, stream)


def qk_norm_rope_backward_workspace(d, device="cuda"):
    """Workspace of qk_norm_rope_backward, for callers that keep one (one for each call that may run at the same time)."""
    import torch
    n = fa_qk_norm_rope_bwd_workspace_bytes(d)
    if n == 0:
        raise FAError(FA_ERR_UNSUPPORTED_HEADDIM, "fa_qk_norm_rope_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, dq_out, dk_out,
                           dq_weight, dk_weight, workspace, stream):
    (B, Hq, N, d), dev, code, dt = _first(q, "q", 4, "[B, Hq, N, d]")
    qp = _check_view(q, "q", q.shape, dt, dev)
    dqp = _check_view(dq, "dq", (B, Hq, N, d), dt, dev)
    Hk, kp, ks, dkp, dks = 0, None, None, None, None
    if k is not None:
        Hk = k.shape[1] if isinstance(k, _torch.Tensor) and k.dim() == 4 else 0
        kp = _check_view(k, "k", (B, Hk, N, d), dt, dev)
        dkp = _check_view(dk, "dk", (B, Hk, N, d), dt, dev)
        ks, dks = _pack3(*k.stride()[:3]), _pack3(*dk.stride()[:3])
    elif not (dk is None and k_weight is None and dk_out is None and dk_weight is None):
        raise ValueError("dk, k_weight, dk_out or dk_weight without k")
    for w, dw, name in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
        if w is None and dw is not None:
            raise ValueError(f"{name} without its weights")
    norm = _norm(q_weight, k_weight, eps, d, dt, dev)
    rot = _maybe_rotary(positions, inv_freq, axes, interleaved, d, (B, N), dev)
    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved,
                                          dq_out, dk_out, dq_weight, dk_weight, workspace, None)
    dq_out, op, os_ = _rows_like(dq_out, "dq_out", (B, Hq, N, d), dt, dev)
    okp, oks = None, None
    if k is not None:
        dk_out, okp, oks = _rows_like(dk_out, "dk_out", (B, Hk, N, d), dt, dev)
    grads = []
    for w, dw, name in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
        if w is None:
            grads += [None, None]
        elif dw is None:
            dw = _torch.empty((d,), dtype=_torch.float32, device=q.device)
            grads += [dw, dw.data_ptr()]
        else:
            grads += [dw, _check_dense(dw, name, (d,), _torch.float32, dev)]
    wp, n = None, 0
    if grads[1] or grads[3]:
        if workspace is None:
            workspace = qk_norm_rope_backward_workspace(d, q.device)
        n = workspace.numel()
        wp = _check_dense(workspace, "workspace", (n,), _torch.uint8, dev)
    status = fa_qk_norm_rope_bwd(dqp, _pack3(*dq.stride()[:3]), qp, _pack3(*q.stride()[:3]), op, os_, dkp, dks, kp, ks, okp,
                                 oks, grads[1], grads[3], B, Hq, Hk, N, d, code, norm, rot, wp, n, handle)
    if status:
        _raise(status, "fa_qk_norm_rope_bwd")
    return (dq_out, grads[0]) if k is None else (dq_out, dk_out, grads[0], grads[2])


def paged4_cache(pages, Hkv, page_size, d, device="cuda"):
    """A pool for ``paged4_append``: uint8 [pages, Hkv, page_size, d + d/8], K and V in 4 bits.
    Its contents are the library's; whole pages may be copied."""
    import torch
    if d not in (64, 128):
        raise FAError(FA_ERR_UNSUPPORTED_HEADDIM, "paged4_cache")
    if page_size < 16 or page_size > 65536 or page_size % 16:
        raise FAError(FA_ERR_BAD_SHAPE, "paged4_cache")
    return torch.empty((pages, Hkv, page_size, d + d // 8), dtype=torch.uint8, device=device)


def _paged4(cache, block_table, seq_lens, dtype):
    """Checked cache tensors: (Hkv, d, device index, fa_paged4_kv, fa_page_table, B, seq_lens address)."""
    if _torch is None:
        _load_torch()
    if not isinstance(cache, _torch.Tensor):
        raise TypeError("cache must be a torch.Tensor")
    if cache.dim() != 4 or cache.shape[3] not in (72, 144):
        raise ValueError(f"cache must be a [pages, Hkv, page_size, d + d/8] tensor with d 64 or 128, got shape "
                         f"{tuple(cache.shape)}")
    code = {_torch.bfloat16: FA_BF16, _torch.float16: FA_FP16}.get(dtype)
    if code is None:
        raise TypeError(f"the cache's values must be torch.bfloat16 or torch.float16, got {dtype}")
    dev = cache.get_device()
    if not cache.is_cuda:
        raise ValueError(f"cache must be a CUDA tensor, got {cache.device}")
    p = _check_view(cache, "cache", cache.shape, _torch.uint8, dev)
    (P, Hkv, ps, row), st = cache.shape, cache.stride()
    if ps > 1 and st[2] != row:
        raise ValueError("cache must be contiguous in its last two dimensions")
    d = row // 9 * 8
    table, B = _table(block_table, "block_table", dev)
    return (Hkv, d, dev, _pack_kv4(p, st[0], st[1], P, ps, Hkv, d, code), table, B,
            _check_dense(seq_lens, "seq_lens", (B,), _torch.int32, dev))


def paged4_append(cache, block_table, seq_lens, k, v, cu_seqlens=None, q=None, q_weight=None, k_weight=None,
                  eps: float | None = None, positions=None, inv_freq=None, axes=None, interleaved: bool = False, q_out=None,
                  stream=None):
    """``paged_append`` into a cache of ``paged4_cache``: k, v [T,Hkv,d] are stored in 4
    bits.  With ``eps`` k, and q [T,Hq,d] if given, are normed first (weights as in
    ``qk_norm_rope``); with ``positions`` [n_axes,T], ``inv_freq`` and ``axes`` they are
    then turned.  Returns q so (into ``q_out``, which may be q), or None without q.
    A cache's calls must all have the same type.  See fa_paged4_append."""
    if stream is None:
        r = (_native or _load_native()).paged4_append(cache, block_table, seq_lens, k, v, cu_seqlens, q, q_weight, k_weight, eps,
                                                      positions, inv_freq, axes, interleaved, q_out)
        if r is not None:
            return None if r is False else _answer(r, "fa_paged4_append")
    return _paged4_append(cache, block_table, seq_lens, k, v, cu_seqlens, q, q_weight, k_weight, eps, positions, inv_freq,
                          axes, interleaved, q_out, stream)


def _paged4_append(cache, block_table, seq_lens, k, v, cu_seqlens, q, q_weight, k_weight, eps, positions, inv_freq, axes,
                   interleaved, q_out, stream):
    if _torch is None:
        _load_torch()
    if not isinstance(k, _torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    dt = k.dtype
    Hkv, d, dev, kv, table, B, lens = _paged4(cache, block_table, seq_lens, dt)
    T = k.shape[0] if k.dim() == 3 else 0
    kp = _check_view(k, "k", (T, Hkv, d), dt, dev)
    vp = _check_view(v, "v", (T, Hkv, d), dt, dev)
    if cu_seqlens is None:
        cu = None
        if T != B:
            raise ValueError(f"{T} tokens for {B} sequences without cu_seqlens")
    else:
        cu = _check_dense(cu_seqlens, "cu_seqlens", (B + 1,), _torch.int32, dev)
    norm = None
    if eps is not None:
        norm = _norm(q_weight, k_weight, eps, d, dt, dev)
    elif q_weight is not None or k_weight is not None:
        raise ValueError("weights of a norm without eps")
    rot = _maybe_rotary(positions, inv_freq, axes, interleaved, d, (T,), dev)
    qp, qs, Hq = None, None, 0
    if q is not None:
        if norm is None and rot is None:
            raise ValueError("q without a norm or a rotation")
        Hq = q.shape[1] if isinstance(q, _torch.Tensor) and q.dim() == 3 else 0
        qp = _check_view(q, "q", (T, Hq, d), dt, dev)
        qs = _pack2(*q.stride()[:2])
    elif q_out is not None:
        raise ValueError("q_out without q")
    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _paged4_append(cache, block_table, seq_lens, k, v, cu_seqlens, q, q_weight, k_weight, eps, positions,
                                  inv_freq, axes, interleaved, q_out, None)
    op, os_ = None, None
    if q is not None:
        q_out, op, os_ = _rows_like(q_out, "q_out", (T, Hq, d), dt, dev)
    if T:
        status = fa_paged4_append(kv, table, lens, cu, B, T, kp, _pack2(*k.stride()[:2]), vp, _pack2(*v.stride()[:2]), qp,
                                  qs, op, os_, Hq, norm, rot, handle)
        if status:
            _raise(status, "fa_paged4_append")
    return q_out


def paged4_read(cache, block_table, seq_lens, n: int, dtype, k_out=None, v_out=None, stream=None):
    """The last n keys of each sequence of a 4-bit cache as k, v [B,Hkv,n,d] of
    ``dtype``, the type it was appended in; row i is key seq_lens[b] - n + i, zero
    where that is negative.  With one sequence's whole length they are, in bf16,
    what ``forward_ex`` (bf16 only) takes for its next queries.  See
    fa_paged4_read."""
    if stream is None:
        r = (_native or _load_native()).paged4_read(cache, block_table, seq_lens, n, dtype, k_out, v_out)
        if r is not None:
            return _answer(r, "fa_paged4_read")
    return _paged4_read(cache, block_table, seq_lens, n, dtype, k_out, v_out, stream)


def _paged4_read(cache, block_table, seq_lens, n, dtype, k_out, v_out, stream):
    Hkv, d, dev, kv, table, B, lens = _paged4(cache, block_table, seq_lens, dtype)
    if n < 1:
        raise ValueError("n must be at least 1")
    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _paged4_read(cache, block_table, seq_lens, n, dtype, k_out, v_out, None)
    k_out, kp, ks = _rows_like(k_out, "k_out", (B, Hkv, n, d), dtype, dev)
    v_out, vp, vs = _rows_like(v_out, "v_out", (B, Hkv, n, d), dtype, dev)
    status = fa_paged4_read(kv, table, lens, kp, ks, vp, vs, B, n, handle)
    if status:
        _raise(status, "fa_paged4_read")
    return k_out, v_out


_decode4_ws_bytes = functools.lru_cache(maxsize=256)(
    lambda *shape: fa_paged4_decode_workspace_bytes(*shape))


def paged4_decode_workspace(B, Hq, cache):
    """Workspace of paged4_decode, for callers that keep one (one for each call that may run at the same time)."""
    import torch
    n = _decode4_ws_bytes(B, Hq, cache.shape[1], cache.shape[3] // 9 * 8)
    if n == 0:
        raise FAError(FA_ERR_BAD_SHAPE, "fa_paged4_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def paged4_decode(q, cache, block_table, seq_lens, scale: float | None = None, window: int = 0, out=None, lse=None,
                  workspace=None, stream=None):
    """O [B,Hq,d], LSE [B,Hq] of one query row per sequence, q [B,Hq,d], against the
    seq_lens[b] keys of a 4-bit cache (the last ``window`` of them if window > 0),
    as the values that it holds.  See fa_paged4_decode."""
    if stream is None:
        r = (_native or _load_native()).paged4_decode(q, cache, block_table, seq_lens, scale, window, out, lse, workspace)
        if r is not None:
            return _answer(r, "fa_paged4_decode")
    return _paged4_decode(q, cache, block_table, seq_lens, scale, window, out, lse, workspace, stream)


def _paged4_decode(q, cache, block_table, seq_lens, scale, window, out, lse, workspace, stream):
    (B, Hq, _), _, _, dt = _first(q, "q", 3, "[B, Hq, d]")
    Hkv, d, dev, kv, table, rows, lens = _paged4(cache, block_table, seq_lens, dt)
    qp = _check_view(q, "q", (rows, Hq, d), dt, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    handle = _raw_stream(dev, stream)
    if handle is None:
        with _on(dev, stream):
            return _paged4_decode(q, cache, block_table, seq_lens, scale, window, out, lse, workspace, None)
    if out is None:
        out = _torch.empty((B, Hq, d), dtype=dt, device=cache.device)
    op = _check_dense(out, "out", (B, Hq, d), dt, dev)
    if lse is None:
        lse = _torch.empty((B, Hq), dtype=_torch.float32, device=cache.device)
    lp = _check_dense(lse, "lse", (B, Hq), _torch.float32, dev)
    if workspace is None:
        workspace = paged4_decode_workspace(B, Hq, cache)
    n = workspace.numel()
    wp = _check_dense(workspace, "workspace", (n,), _torch.uint8, dev)
    status = fa_paged4_decode(qp, _pack2(*q.stride()[:2]), kv, table, lens, op, lp, B, Hq, window, scale, wp, n, handle)
    if status:
        _raise(status, "fa_paged4_decode")
    return out, lse

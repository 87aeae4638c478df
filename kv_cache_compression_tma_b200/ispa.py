"""ctypes binding of libispa.so (the C ABI in include/ispa.h).

Argument marshalling only: every step of the hot path runs in the library's CUDA kernels.  PyTorch
provides device memory and the current stream.  If the library is missing the calls raise; there
is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libispa.so")

ISPA_OK, ISPA_ERR_INVALID_ARG, ISPA_ERR_UNSUPPORTED, ISPA_ERR_CUDA = 0, 1, 2, 3
ISPA_ERR_NOT_SPD, ISPA_ERR_NONFINITE, ISPA_ERR_TIMEOUT, ISPA_ERR_INTERNAL = 4, 5, 6, 7
ISPA_BF16, ISPA_F32 = 0, 1
ISPA_ATTN_CUDA_CORES = 0x1
ISPA_STATS_ZERO, ISPA_STATS_SECOND_IS_FULL = 0x1, 0x2
ISPA_LAMBDA_REL, ISPA_W_TRANSPOSED, ISPA_WRITE_WNEW = 0x1, 0x2, 0x4
ISPA_TEST_ATTN_NO_LOADS = 0x1
ISPA_QUANT_COLUMNS = 0x1

SYMBOLS = ("ispa_dual_stream_attn", "ispa_accum_stats", "ispa_absorb_workspace_size", "ispa_absorb",
           "ispa_absorb_static", "ispa_project", "ispa_quantize_e4m3", "ispa_project_w8a8", "ispa_tempcache_match",
           "ispa_tempcache_merge", "ispa_attn_mass", "ispa_cache_insert", "ispa_block_means", "ispa_block_select",
           "ispa_block_sparse_attn", "ispa_select_layers",
           "ispa_get_device_status",
           "ispa_peek_device_status_bits", "ispa_test_set_flags",
           "ispa_status_string", "ispa_version", "ispa_launch_count")


class IspaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class AttnArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("flags", ctypes.c_int32), ("n_q", ctypes.c_int64), ("n_kv", ctypes.c_int64 * 3),
        ("q", ctypes.c_void_p), ("ld_q", ctypes.c_int64),
        ("k", ctypes.c_void_p * 3), ("v", ctypes.c_void_p * 3),
        ("ld_k", ctypes.c_int64 * 3), ("ld_v", ctypes.c_int64 * 3),
        ("softmax_scale", ctypes.c_float), ("reserved0", ctypes.c_float),
        ("o_loc", ctypes.c_void_p), ("o_full", ctypes.c_void_p), ("ld_o", ctypes.c_int64),
        ("lse_loc", ctypes.c_void_p), ("lse_hist", ctypes.c_void_p), ("d_out", ctypes.c_void_p),
        ("kv_bias", ctypes.c_void_p * 3), ("ld_bias", ctypes.c_int64 * 3),
    ]


# AttnArgs' fields for the calls of single tokens: packing them takes a microsecond, filling the structure five.
_ATTN_ARGS = struct.Struct("4iq3qQq3Q3Q3q3q2fQQqQQQ3Q3q")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libispa.so (built in-tree by kv_cache_compression_tma_b200.build); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m kv_cache_compression_tma_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.ispa_dual_stream_attn.argtypes = [ctypes.POINTER(AttnArgs), ctypes.c_void_p]
        L.ispa_accum_stats.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.ispa_absorb_workspace_size.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
        L.ispa_absorb.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                  ctypes.c_int32, ctypes.c_float, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.ispa_absorb_static.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                         ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_uint32,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.ispa_project.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int64,
                                   ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p,
                                   ctypes.c_int64, ctypes.c_void_p]
        L.ispa_quantize_e4m3.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                         ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_void_p]
        L.ispa_project_w8a8.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
        L.ispa_tempcache_match.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p]
        L.ispa_tempcache_merge.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p]
        c32, c64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        L.ispa_attn_mass.argtypes = [c32, c32, c32, vp, c64, c64, vp, c64, c64, vp, vp, vp, c64, ctypes.c_float,
                                     ctypes.c_float, ctypes.c_uint32, vp, vp, c64, vp]
        L.ispa_cache_insert.argtypes = [c32, c32, c32, vp, vp, c64, c64, c64, vp, vp, c64, vp, vp, c64, c64, vp, c64,
                                        c32, c32, c32, vp, vp, c64, vp]
        L.ispa_block_means.argtypes = [c32, c32, c32, vp, c64, c64, c32, c64, vp, c64, vp]
        L.ispa_block_select.argtypes = [c32, c32, c32, vp, c64, c64, c32, vp, c64, c64, c32, vp, vp]
        L.ispa_block_sparse_attn.argtypes = [vp, vp, c32, c32, c32, vp]
        L.ispa_select_layers.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.c_int32, ctypes.c_int32,
                                         ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_uint8)]
        L.ispa_get_device_status.argtypes = [ctypes.c_void_p]
        L.ispa_peek_device_status_bits.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        L.ispa_test_set_flags.argtypes = [ctypes.c_uint32]
        L.ispa_status_string.argtypes = [ctypes.c_int32]
        L.ispa_status_string.restype = ctypes.c_char_p
        L.ispa_version.restype = ctypes.c_int32
        L.ispa_launch_count.restype = ctypes.c_uint64
        for name in ("ispa_dual_stream_attn", "ispa_accum_stats", "ispa_absorb_workspace_size", "ispa_absorb",
                     "ispa_absorb_static", "ispa_select_layers", "ispa_get_device_status", "ispa_peek_device_status_bits",
                     "ispa_test_set_flags", "ispa_quantize_e4m3", "ispa_project_w8a8", "ispa_tempcache_match",
                     "ispa_tempcache_merge", "ispa_attn_mass", "ispa_cache_insert", "ispa_block_means",
                     "ispa_block_select", "ispa_block_sparse_attn"):
            getattr(L, name).restype = ctypes.c_int32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ispa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != ISPA_OK:
        raise IspaError(status, what)


def _stream(stream=None) -> int:
    import torch
    if stream is None:  # the raw handle: a Stream object costs several microseconds per call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return int(stream.cuda_stream)


def _alloc_on(stream):
    """Where a call on `stream` allocates what it returns or drops: from that stream's memory, whose reuse
    follows the call's kernels."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return ISPA_BF16
    if t.dtype == torch.float32:
        return ISPA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _on_current_device(*tensors):
    """The library resolves its per-device state (status word, scratch, streams) from the CURRENT
    device, so every tensor of a call must live there."""
    import torch
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:  # -1 for a host tensor
            raise ValueError(f"tensor on {t.device}, but the current CUDA device is cuda:{cur}; "
                             f"call under `with torch.cuda.device(...)`")


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _row_stride(t, what: str) -> int:
    """Token/row stride of a [tokens, H, hd] or [rows, d] tensor whose inner dims are dense."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        if stride[2] != 1 or stride[1] != shape[2]:
            raise ValueError(f"{what}: heads and head_dim must be contiguous")
    elif len(shape) == 2:
        if stride[1] != 1:
            raise ValueError(f"{what}: columns must be contiguous")
    else:
        raise ValueError(f"{what}: expected 2 or 3 dims")
    if shape[0] <= 1:  # a single row: its stride is irrelevant, report the dense row length
        return math.prod(shape[1:])
    return stride[0]


def _heads_rows(t, what: str, H: int, hd: int, dtype, device: int, n: Optional[int] = None):
    """(tokens, token stride) of a [tokens, H, hd] tensor of this type on the current device whose heads
    and head_dim are dense; n: how many tokens it must have."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != H or shape[2] != hd or t.dtype != dtype or (n is not None and shape[0] != n):
        raise ValueError(f"{what}: expected {dtype} [{'tokens' if n is None else n}, {H}, {hd}]")
    if t.get_device() != device:
        _on_current_device(t)
    stride = t.stride()
    if stride[2] != 1 or (stride[1] != hd and H > 1):
        raise ValueError(f"{what}: heads and head_dim must be contiguous")
    return shape[0], stride[0] if shape[0] > 1 else H * hd


INT32_MAX = 2 ** 31 - 1


def _int32(x: int, what: str, low: int = -2 ** 31) -> int:
    """x as the ABI's int32: ctypes would drop the high bits of a larger one without a word."""
    if not low <= x <= INT32_MAX:
        raise ValueError(f"{what} must lie in {low} .. 2^31 - 1")
    return x


def _pieces(n: int, size: int, what: str) -> int:
    """How many pieces of `size` cover n."""
    return -(-n // _int32(size, what, 1))


def _state_rows(t, what: str, H: int, cols: int, dtype, device: int) -> int:
    """Row stride of a per-head array [H, >= cols] of this type on the current device, columns contiguous; a
    lone head's row has none, and the largest length stands for it in every array."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != H or shape[1] < cols or t.dtype != dtype or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what}: expected {dtype} [{H}, >= {cols}] with contiguous columns")
    if t.get_device() != device:
        _on_current_device(t)
    return stride[0] if H > 1 else 1 << 30


def _dense(t, what: str, shape, dtype, device: int) -> int:
    """Address of a contiguous array of this shape and type on the current device."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {dtype} {list(shape)}")
    if t.get_device() != device:
        _on_current_device(t)
    return t.data_ptr()


def dual_stream_attn(q, k_sink, v_sink, k_loc, v_loc, k_hist, v_hist, *, o_loc=None, o_full=None, lse_loc=None,
                     lse_hist=None, d_out=None, want_delta: bool = True, softmax_scale: float = 0.0,
                     cuda_cores: bool = False, kv_bias=(None, None, None), stream=None) -> dict:
    """ispa_dual_stream_attn on torch CUDA tensors.

    q, k_*, v_*: [tokens, H, hd] (bf16 or fp32).  Outputs (allocated if not given): o_loc, o_full and
    (if want_delta) d = O_full - O_loc as [n_q, H*hd] in q's dtype; lse_loc, lse_hist fp32 [H, n_q].
    kv_bias: optional per-segment fp32 [H, n_kv] additive logit biases (natural log), e.g. the log group
    sizes of a TempCache-merged history.
    """
    import torch
    _on_current_device(q, k_sink, v_sink, k_loc, v_loc, k_hist, v_hist, o_loc, o_full, lse_loc, lse_hist, d_out,
                       *kv_bias)
    n_q, H, hd = q.shape
    d = H * hd
    dev = q.device
    with _alloc_on(stream):
        if o_loc is None:
            o_loc = torch.empty((n_q, d), dtype=q.dtype, device=dev)
        if o_full is None:
            o_full = torch.empty((n_q, d), dtype=q.dtype, device=dev)
        if d_out is None and want_delta:
            d_out = torch.empty((n_q, d), dtype=q.dtype, device=dev)
        if lse_loc is None:
            lse_loc = torch.empty((H, n_q), dtype=torch.float32, device=dev)
        if lse_hist is None:
            lse_hist = torch.empty((H, n_q), dtype=torch.float32, device=dev)
    n_kv, k_ptr, v_ptr, ld_k, ld_v = [], [], [], [], []
    for k, v in ((k_sink, v_sink), (k_loc, v_loc), (k_hist, v_hist)):
        n = k.shape[0]
        n_kv.append(n)
        k_ptr.append(k.data_ptr() if n else None)
        v_ptr.append(v.data_ptr() if n else None)
        ld_k.append(_row_stride(k, "k") if n else d)
        ld_v.append(_row_stride(v, "v") if n else d)
    bias, ld_bias = [None] * 3, [0] * 3
    for i, bt in enumerate(kv_bias):
        if bt is not None:
            if bt.dtype != torch.float32 or bt.dim() != 2 or bt.stride(1) != 1:
                raise ValueError("kv_bias entries must be fp32 [H, n_kv] with contiguous columns")
            bias[i], ld_bias[i] = bt.data_ptr(), bt.stride(0)
    a = AttnArgs(_dtype_code(q), H, hd, ISPA_ATTN_CUDA_CORES if cuda_cores else 0, n_q, tuple(n_kv), q.data_ptr(),
                 _row_stride(q, "q") if n_q else d, tuple(k_ptr), tuple(v_ptr), tuple(ld_k), tuple(ld_v),
                 softmax_scale, 0.0, o_loc.data_ptr(), o_full.data_ptr(), _row_stride(o_loc, "o_loc") if n_q else d,
                 lse_loc.data_ptr(), lse_hist.data_ptr(), _ptr(d_out), tuple(bias), tuple(ld_bias))
    _check(lib().ispa_dual_stream_attn(ctypes.byref(a), _stream(stream)), "ispa_dual_stream_attn")
    return {"o_loc": o_loc, "o_full": o_full, "d": d_out, "lse_loc": lse_loc, "lse_hist": lse_hist}


def accum_stats(a_loc, a_second, G, R, S, *, second_is_full: bool = False, zero: bool = False, stream=None):
    """ispa_accum_stats: G/R/S (fp32 [d, d]) (+)= A_loc^T A_loc, A_loc^T D, D^T D over the rows given."""
    _on_current_device(a_loc, a_second, G, R, S)
    m, d = a_loc.shape
    flags = (ISPA_STATS_ZERO if zero else 0) | (ISPA_STATS_SECOND_IS_FULL if second_is_full else 0)
    lda = _row_stride(a_loc, "a_loc") if m else d
    if m and _row_stride(a_second, "a_second") != lda:
        raise ValueError("a_loc and a_second must share a row stride")
    _check(lib().ispa_accum_stats(_dtype_code(a_loc), _ptr(a_loc), _ptr(a_second), m, d, lda, flags, _ptr(G),
                                  _ptr(R), _ptr(S), _stream(stream)), "ispa_accum_stats")
    return G, R, S


def absorb_workspace_size(d: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ispa_absorb_workspace_size(int(d), ctypes.byref(n)), "ispa_absorb_workspace_size")
    return int(n.value)


def absorb(G, R, S, W, lam: float, *, lam_rel: bool = False, w_transposed: bool = False, dW=None, eps=None,
           w_new=None, write_wnew: bool = False, ws=None, stream=None) -> dict:
    """ispa_absorb: dW = (G + lam I)^-1 R W and eps = {eps, eps_rel, lam, <W, S W>} (fp64, on device)."""
    import torch
    _on_current_device(G, R, S, W, dW, eps, w_new, ws)
    d = G.shape[0]
    dev = G.device
    with _alloc_on(stream):
        if dW is None:
            dW = torch.empty((d, d), dtype=torch.float32, device=dev)
        if eps is None:
            eps = torch.empty((4,), dtype=torch.float64, device=dev)
        if ws is None:
            ws = torch.empty((absorb_workspace_size(d),), dtype=torch.uint8, device=dev)
        if write_wnew and w_new is None:
            w_new = torch.empty_like(W)
    flags = (ISPA_LAMBDA_REL if lam_rel else 0) | (ISPA_W_TRANSPOSED if w_transposed else 0) | \
            (ISPA_WRITE_WNEW if write_wnew else 0)
    _check(lib().ispa_absorb(_ptr(G), _ptr(R), _ptr(S), _dtype_code(W), _ptr(W), d, float(lam), flags, _ptr(dW),
                             _ptr(eps), _ptr(w_new), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "ispa_absorb")
    return {"dW": dW, "eps": eps, "w_new": w_new, "ws": ws}


ABSORB_STATIC_MAX_D = 1536


def absorb_static(G, R, S, W, lam: float, *, lam_rel: bool = False, w_transposed: bool = False, dW=None,
                  eps=None, w_new=None, write_wnew: bool = False, stream=None) -> dict:
    """ispa_absorb_static: the absorb without a caller workspace (library-held scratch, d <= 1536).
    For callers that cannot allocate device memory at absorb time; the outputs are still the caller's."""
    import torch
    _on_current_device(G, R, S, W, dW, eps, w_new)
    d = G.shape[0]
    dev = G.device
    with _alloc_on(stream):
        if dW is None:
            dW = torch.empty((d, d), dtype=torch.float32, device=dev)
        if eps is None:
            eps = torch.empty((4,), dtype=torch.float64, device=dev)
        if write_wnew and w_new is None:
            w_new = torch.empty_like(W)
    flags = (ISPA_LAMBDA_REL if lam_rel else 0) | (ISPA_W_TRANSPOSED if w_transposed else 0) | \
            (ISPA_WRITE_WNEW if write_wnew else 0)
    _check(lib().ispa_absorb_static(_ptr(G), _ptr(R), _ptr(S), _dtype_code(W), _ptr(W), d, float(lam), flags,
                                    _ptr(dW), _ptr(eps), _ptr(w_new), _stream(stream)), "ispa_absorb_static")
    return {"dW": dW, "eps": eps, "w_new": w_new}


def project(A, W, *, w_transposed: bool = False, out=None, stream=None):
    """ispa_project: Y = A W (or A W^T for a torch-Linear-layout W) with A [m, d_in] and W [d_in, d_out]
    ([d_out, d_in] when w_transposed); bf16 runs the tensor-core kernel, fp32 the CUDA-core one."""
    import torch
    _on_current_device(A, W, out)
    if A.dtype != W.dtype:
        raise ValueError("A and W must have the same dtype")
    m, d_in = A.shape
    d_out = W.shape[0] if w_transposed else W.shape[1]
    if (W.shape[1] if w_transposed else W.shape[0]) != d_in:
        raise ValueError("W does not match A's width")
    if out is None:
        with _alloc_on(stream):
            out = torch.empty((m, d_out), dtype=A.dtype, device=A.device)
    flags = ISPA_W_TRANSPOSED if w_transposed else 0
    _check(lib().ispa_project(_dtype_code(A), _ptr(A), m, d_in, _row_stride(A, "A"), _ptr(W), d_out,
                              _row_stride(W, "W"), flags, _ptr(out), _row_stride(out, "out"), _stream(stream)),
           "ispa_project")
    return out


def quantize_e4m3(X, *, columns: bool = False, q=None, scale=None, stream=None):
    """ispa_quantize_e4m3: fp8 E4M3 codes (torch.uint8) and fp32 scales of X [rows, cols] (bf16 or
    fp32).  Per row by default: q [rows, cols], scale [rows].  columns=True: per column, q written
    transposed [cols, rows] (the K-major weight layout of project_w8a8), scale [cols]."""
    import torch
    _on_current_device(X, q, scale)
    rows, cols = X.shape
    with _alloc_on(stream):
        if q is None:
            q = torch.empty((cols, rows) if columns else (rows, cols), dtype=torch.uint8, device=X.device)
        if scale is None:
            scale = torch.empty((cols if columns else rows,), dtype=torch.float32, device=X.device)
    ldx = _row_stride(X, "X") if rows else cols
    ldq = _row_stride(q, "q") if q.shape[0] > 1 else q.shape[1]
    _check(lib().ispa_quantize_e4m3(_dtype_code(X), _ptr(X), rows, cols, ldx, ISPA_QUANT_COLUMNS if columns else 0,
                                    _ptr(q), ldq, _ptr(scale), _stream(stream)), "ispa_quantize_e4m3")
    return q, scale


def project_w8a8(qa, sa, qw, sw, *, out=None, stream=None):
    """ispa_project_w8a8: Y = diag(sa) (qa qw^T) diag(sw) in bf16, with qa [m, d_in] and qw [d_out, d_in]
    E4M3 codes (torch.uint8) from quantize_e4m3."""
    import torch
    _on_current_device(qa, sa, qw, sw, out)
    m, d_in = qa.shape
    d_out = qw.shape[0]
    if qw.shape[1] != d_in:
        raise ValueError("qw does not match qa's width")
    if out is None:
        with _alloc_on(stream):
            out = torch.empty((m, d_out), dtype=torch.bfloat16, device=qa.device)
    _check(lib().ispa_project_w8a8(_ptr(qa), _ptr(sa), m, d_in, _row_stride(qa, "qa"), _ptr(qw), _ptr(sw), d_out,
                                   _row_stride(qw, "qw"), _ptr(out), _row_stride(out, "out"), _stream(stream)),
           "ispa_project_w8a8")
    return out


class TempCache:
    """A TempCache-merged KV segment on the device (FAST-AR TempCache): per-head entries with
    representative keys, mean values, group sizes, their logs as the attention bias, and inverse key
    norms; see ispa_tempcache_match / ispa_tempcache_merge in include/ispa.h."""

    def __init__(self, n_heads: int, head_dim: int, capacity: int, device="cuda"):
        import torch
        self.n_heads, self.head_dim, self.capacity = n_heads, head_dim, capacity
        ld_state = (capacity + 3) // 4 * 4
        self.k = torch.zeros((capacity, n_heads, head_dim), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.count = torch.zeros((n_heads, ld_state), dtype=torch.int32, device=device)
        self.bias = torch.full((n_heads, ld_state), float("-inf"), dtype=torch.float32, device=device)
        self.inv_norm = torch.full((n_heads, ld_state), -1.0, dtype=torch.float32, device=device)
        self.n_valid = torch.zeros((n_heads,), dtype=torch.int32, device=device)
        self.n_cache = 0  # bound on every head's entry count: the segment length to attend over

    def match(self, k_new, idx=None, sim=None, stream=None):
        import torch
        _on_current_device(k_new, self.k, idx, sim)
        n_new = k_new.shape[0]
        with _alloc_on(stream):
            if idx is None:
                idx = torch.empty((self.n_heads, n_new), dtype=torch.int32, device=k_new.device)
            if sim is None:
                sim = torch.empty((self.n_heads, n_new), dtype=torch.float32, device=k_new.device)
        ld_new = _row_stride(k_new, "k_new") if n_new else self.n_heads * self.head_dim
        _check(lib().ispa_tempcache_match(self.n_heads, self.head_dim, _ptr(k_new), n_new, ld_new, _ptr(self.k),
                                          self.n_cache, self.n_heads * self.head_dim, _ptr(self.inv_norm),
                                          self.count.stride(0), _ptr(idx), _ptr(sim), _stream(stream)),
               "ispa_tempcache_match")
        return idx, sim

    def merge(self, k_new, v_new, idx, sim, threshold: float, stream=None):
        _on_current_device(k_new, v_new, idx, sim, self.k)
        n_new = k_new.shape[0]
        ld_new = _row_stride(k_new, "k_new") if n_new else self.n_heads * self.head_dim
        if n_new and _row_stride(v_new, "v_new") != ld_new:
            raise ValueError("k_new and v_new must share a row stride")
        _check(lib().ispa_tempcache_merge(self.n_heads, self.head_dim, _ptr(self.k), _ptr(self.v),
                                          self.n_heads * self.head_dim, self.capacity, self.n_cache, _ptr(self.count),
                                          _ptr(self.bias), _ptr(self.inv_norm), self.count.stride(0),
                                          _ptr(self.n_valid), _ptr(k_new), _ptr(v_new), n_new, ld_new, _ptr(idx),
                                          _ptr(sim), float(threshold), _stream(stream)), "ispa_tempcache_merge")
        self.n_cache += n_new

    def add_frame(self, k_new, v_new, threshold: float, stream=None):
        """Match then merge one frame; returns (idx, sim) of the match."""
        idx, sim = self.match(k_new, stream=stream)
        self.merge(k_new, v_new, idx, sim, threshold, stream=stream)
        return idx, sim

    def segment(self):
        """(k, v, bias) views of the live bound, for dual_stream_attn's history segment."""
        n = self.n_cache
        return self.k[:n], self.v[:n], self.bias[:, :n]


def attn_mass(q, k, lse_loc, lse_hist, mass, *, kv_bias=None, decay: float = 1.0, softmax_scale: float = 0.0,
              cuda_cores: bool = False, mass_out=None, stream=None):
    """ispa_attn_mass: mass[h, j] = decay * mass[h, j] + the attention weight that key j collects from the
    queries q [n_q, H, hd], for the keys k [n_k, H, hd] of one segment.  lse_loc, lse_hist: fp32 [H, n_q],
    contiguous, as dual_stream_attn returned them for the same queries (lse_hist None: no history branch);
    those of block_sparse_attn leave out the keys that were not picked, which may then weigh more than 1.
    kv_bias: fp32 [H, >= n_k], the segment's bias in that call.  mass fp32 [H, >= n_k]; the result goes to
    mass_out (same shape and stride as mass) or back into mass.  Returns the array written."""
    import torch
    f32, dev = torch.float32, torch.cuda.current_device()
    n_q, H, hd = q.shape
    dtype = q.dtype
    _, ld_q = _heads_rows(q, "q", H, hd, dtype, dev)
    n_k, ld_k = _heads_rows(k, "k", H, hd, dtype, dev)
    ll = _dense(lse_loc, "lse_loc", (H, n_q), f32, dev)
    lh = None if lse_hist is None else _dense(lse_hist, "lse_hist", (H, n_q), f32, dev)
    ld_mass = _state_rows(mass, "mass", H, n_k, f32, dev)
    if mass_out is None:
        mass_out = mass
    elif _state_rows(mass_out, "mass_out", H, n_k, f32, dev) != ld_mass:
        raise ValueError("mass and mass_out must share a row stride")
    bias, ld_bias = (None, 0) if kv_bias is None else (kv_bias.data_ptr(), _state_rows(kv_bias, "kv_bias", H, n_k, f32, dev))
    _check(lib().ispa_attn_mass(_dtype_code(q), H, hd, q.data_ptr(), n_q, ld_q, k.data_ptr(), n_k, ld_k, ll, lh, bias,
                                ld_bias, softmax_scale, decay, ISPA_ATTN_CUDA_CORES if cuda_cores else 0,
                                mass.data_ptr(), mass_out.data_ptr(), ld_mass, _stream(stream)), "ispa_attn_mass")
    return mass_out


def cache_insert(k_cache, v_cache, mass, pos, n: int, k_new, v_new, mass_new, pos_new: int, *, keep_below: int = 0,
                 keep_from: int = INT32_MAX, mass_out=None, pos_out=None, stream=None) -> int:
    """ispa_cache_insert: the new tokens k_new, v_new [n_new, H, hd] with weights mass_new (fp32 [H, n_new],
    None = 0) at positions pos_new, pos_new + 1, ... enter the cache k_cache, v_cache [capacity, H, hd] that
    holds n entries per head with weights mass (fp32 [H, >= n]) and positions pos (int32); the entries
    of least weight leave.  Positions below keep_below or from keep_from on are protected.  The state
    goes to mass_out, pos_out or back into mass, pos.  Returns the number of entries held afterwards."""
    import torch
    f32, i32, dev = torch.float32, torch.int32, torch.cuda.current_device()
    capacity, H, hd = k_cache.shape
    dtype = k_cache.dtype
    _, ld_cache = _heads_rows(k_cache, "k_cache", H, hd, dtype, dev)
    n_new, ld_new = _heads_rows(k_new, "k_new", H, hd, dtype, dev)
    if _heads_rows(v_cache, "v_cache", H, hd, dtype, dev, capacity)[1] != ld_cache or \
            _heads_rows(v_new, "v_new", H, hd, dtype, dev, n_new)[1] != ld_new:
        raise ValueError("k and v must share a row stride")
    total = min(capacity, n + n_new)
    ld_state = _state_rows(mass, "mass", H, n, f32, dev)
    ld_out = ld_state
    same = _state_rows(pos, "pos", H, n, i32, dev) == ld_state
    if mass_out is None:
        mass_out = mass
    else:
        ld_out = _state_rows(mass_out, "mass_out", H, total, f32, dev)
    if pos_out is None:
        pos_out = pos
    else:
        same = same and _state_rows(pos_out, "pos_out", H, total, i32, dev) == ld_out
    if not same:
        raise ValueError("mass and pos (mass_out and pos_out) must share a row stride")
    if mass.shape[1] < total and mass_out is mass or pos.shape[1] < total and pos_out is pos:
        raise ValueError(f"mass and pos need room for {total} entries per head")
    mn, ld_mn = (None, 0) if mass_new is None else (mass_new.data_ptr(), _state_rows(mass_new, "mass_new", H, n_new, f32, dev))
    _check(lib().ispa_cache_insert(_dtype_code(k_cache), H, hd, k_cache.data_ptr(), v_cache.data_ptr(), ld_cache, capacity,
                                   n, mass.data_ptr(), pos.data_ptr(), ld_state, k_new.data_ptr(), v_new.data_ptr(),
                                   n_new, ld_new, mn, ld_mn, _int32(pos_new, "pos_new"), _int32(keep_below, "keep_below"),
                                   _int32(keep_from, "keep_from"), mass_out.data_ptr(),
                                   pos_out.data_ptr(), ld_out, _stream(stream)), "ispa_cache_insert")
    return total


class MassCache:
    """A KV segment of at most `capacity` entries per head, kept by accumulated attention weight: every
    attention call over it may add the weights its keys collected (accumulate), and new tokens push out
    the entries of least weight (insert); see ispa_attn_mass / ispa_cache_insert in include/ispa.h."""

    def __init__(self, n_heads: int, head_dim: int, capacity: int, dtype=None, device="cuda"):
        import torch
        self.n_heads, self.head_dim, self.capacity = n_heads, head_dim, capacity
        self.k = torch.zeros((capacity, n_heads, head_dim), dtype=dtype or torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.mass = torch.zeros((n_heads, capacity), dtype=torch.float32, device=device)
        self.pos = torch.zeros((n_heads, capacity), dtype=torch.int32, device=device)
        self.n = 0     # entries held, the same for every head
        self.seen = 0  # tokens inserted so far: the next token's position

    def segment(self):
        """(k, v) views of the held entries, for dual_stream_attn's history segment.  insert replaces entries in
        place, so what is kept about these keys (a BlockIndex's means) holds until the next insert only."""
        return self.k[:self.n], self.v[:self.n]

    def accumulate(self, q, lse_loc, lse_hist=None, *, decay: float = 1.0, softmax_scale: float = 0.0, stream=None):
        """Add the weights that the held keys collected from q in the attention call that gave the lse's (over all
        held keys: see attn_mass for lse's that leave some out)."""
        attn_mass(q, self.k[:self.n], lse_loc, lse_hist, self.mass, decay=decay, softmax_scale=softmax_scale,
                  stream=stream)

    def insert(self, k_new, v_new, mass_new=None, *, first: int = 0, recent: int = 0, stream=None):
        """Insert a frame's tokens; the first `first` positions of the stream and its newest `recent`
        tokens are protected (together at most `capacity`)."""
        if first < 0 or recent < 0 or first + recent > self.capacity:
            raise ValueError(f"first + recent must lie in 0 .. {self.capacity}")
        n_new = k_new.shape[0]
        keep_from = max(0, self.seen + n_new - recent) if recent > 0 else INT32_MAX
        self.n = cache_insert(self.k, self.v, self.mass, self.pos, self.n, k_new, v_new, mass_new, self.seen,
                              keep_below=first, keep_from=keep_from, stream=stream)
        self.seen += n_new


def block_means(k, means, block: int, *, first: int = 0, stream=None):
    """ispa_block_means: means[b] (fp32 [>= blocks, H, hd]) = mean key of block b of k [n_k, H, hd], for the
    blocks from `first` on; earlier rows are left as they are."""
    import torch
    dev = torch.cuda.current_device()
    _, H, hd = k.shape
    n_k, ld_k = _heads_rows(k, "k", H, hd, k.dtype, dev)
    rows, ld_means = _heads_rows(means, "means", H, hd, torch.float32, dev)
    if rows < _pieces(n_k, block, "block"):
        raise ValueError("means has fewer rows than k has blocks")
    _int32(first, "first", 0)
    _check(lib().ispa_block_means(_dtype_code(k), H, hd, k.data_ptr(), n_k, ld_k, block, first, means.data_ptr(),
                                  ld_means, _stream(stream)), "ispa_block_means")
    return means


def block_select(q, means, n_sel: int, *, q_block: int = 1, out=None, stream=None):
    """ispa_block_select: int32 [H, ceil(n_q / q_block), n_sel], the blocks (rows of means, fp32 [blocks, H,
    hd]) of highest (mean query of the group) . (mean key), ascending, -1 where there are fewer."""
    import torch
    dev = torch.cuda.current_device()
    n_q, H, hd = q.shape
    _, ld_q = _heads_rows(q, "q", H, hd, q.dtype, dev)
    n_blocks, ld_means = _heads_rows(means, "means", H, hd, torch.float32, dev)
    shape = (H, _pieces(n_q, q_block, "q_block"), n_sel)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(shape, dtype=torch.int32, device=q.device)
    _check(lib().ispa_block_select(_dtype_code(q), H, hd, q.data_ptr(), n_q, ld_q, q_block, means.data_ptr(), n_blocks,
                                   ld_means, _int32(n_sel, "n_sel"), _dense(out, "out", shape, torch.int32, dev), _stream(stream)),
           "ispa_block_select")
    return out


class BlockIndex:
    """The mean keys of a growing history's blocks, and the selection of blocks by them; see
    ispa_block_means / ispa_block_select in include/ispa.h."""

    def __init__(self, n_heads: int, head_dim: int, max_tokens: int, block: int = 128, device="cuda"):
        import torch
        self.block, self.n = block, 0
        self.means = torch.zeros((_pieces(max_tokens, block, "block"), n_heads, head_dim), dtype=torch.float32, device=device)

    def extend(self, k, stream=None):
        """Pool the blocks of the history k [n, H, hd] that its tokens since the last call touch.  The history
        only grows at its end; reset() starts another.  A MassCache's entries change in place, so its
        segment's views are no such history: pass the MassCache itself, whose blocks are all pooled anew."""
        first = self.n // self.block
        if isinstance(k, MassCache):
            k, first = k.k[:k.n], 0
        elif k.shape[0] < self.n:
            raise ValueError(f"the history had {self.n} tokens and now has {k.shape[0]}: reset() first")
        block_means(k, self.means, self.block, first=first, stream=stream)
        self.n = k.shape[0]

    def reset(self):
        self.n = 0

    def select(self, q, n_sel: int, *, q_block: int = 1, out=None, stream=None):
        """The picks for each group of q_block queries; see block_select."""
        return block_select(q, self.means[:_pieces(self.n, self.block, "block")], n_sel, q_block=q_block, out=out, stream=stream)


def block_sparse_attn(q, k_sink, v_sink, k_loc, v_loc, k_hist, v_hist, idx, *, block: int, q_block: int = 1, o_loc=None,
                      o_full=None, lse_loc=None, lse_hist=None, d_out=None, want_delta: bool = True,
                      softmax_scale: float = 0.0, cuda_cores: bool = False, stream=None) -> dict:
    """ispa_block_sparse_attn: dual_stream_attn whose history branch covers only the blocks (of `block`
    tokens of k_hist, v_hist) listed in idx, int32 [H, ceil(n_q / q_block), n_sel], for each group of
    q_block queries (as block_select gives them).  The same outputs as dual_stream_attn."""
    import torch
    dtype, dev, f32 = q.dtype, torch.cuda.current_device(), torch.float32
    n_q, H, hd = q.shape
    n_q, ld_q = _heads_rows(q, "q", H, hd, dtype, dev)
    ns, ld_ks = _heads_rows(k_sink, "k_sink", H, hd, dtype, dev)
    ld_vs = _heads_rows(v_sink, "v_sink", H, hd, dtype, dev, ns)[1]
    nl, ld_kl = _heads_rows(k_loc, "k_loc", H, hd, dtype, dev)
    ld_vl = _heads_rows(v_loc, "v_loc", H, hd, dtype, dev, nl)[1]
    nh, ld_kh = _heads_rows(k_hist, "k_hist", H, hd, dtype, dev)
    ld_vh = _heads_rows(v_hist, "v_hist", H, hd, dtype, dev, nh)[1]
    shape, ld_o = (n_q, H * hd), H * hd
    if o_loc is not None and n_q > 1:
        ld_o = o_loc.stride()[0]
    with _alloc_on(stream):
        if o_loc is None:
            o_loc = torch.empty(shape, dtype=dtype, device=q.device)
        if o_full is None:
            o_full = torch.empty_strided(shape, (ld_o, 1), dtype=dtype, device=q.device)
        if d_out is None and want_delta:
            d_out = torch.empty_strided(shape, (ld_o, 1), dtype=dtype, device=q.device)
        if lse_loc is None:
            lse_loc = torch.empty((H, n_q), dtype=f32, device=q.device)
        if lse_hist is None:
            lse_hist = torch.empty((H, n_q), dtype=f32, device=q.device)
    for o in (o_loc, o_full, d_out):
        if o is None:
            continue
        if o.shape != shape or o.dtype != dtype or o.stride()[1] != 1 or (n_q > 1 and o.stride()[0] != ld_o):
            raise ValueError(f"outputs must be {dtype} {list(shape)} with one row stride")
        if o.get_device() != dev:
            _on_current_device(o)
    n_sel, groups = _int32(idx.shape[-1], "n_sel"), _pieces(n_q, q_block, "q_block")
    a = _ATTN_ARGS.pack(_dtype_code(q), H, hd, ISPA_ATTN_CUDA_CORES if cuda_cores else 0, n_q, ns, nl, nh, q.data_ptr(), ld_q,
                        k_sink.data_ptr(), k_loc.data_ptr(), k_hist.data_ptr(),
                        v_sink.data_ptr(), v_loc.data_ptr(), v_hist.data_ptr(), ld_ks, ld_kl, ld_kh, ld_vs, ld_vl, ld_vh,
                        softmax_scale, 0.0, o_loc.data_ptr(), o_full.data_ptr(), ld_o,
                        _dense(lse_loc, "lse_loc", (H, n_q), f32, dev), _dense(lse_hist, "lse_hist", (H, n_q), f32, dev),
                        0 if d_out is None else d_out.data_ptr(), 0, 0, 0, 0, 0, 0)
    _check(lib().ispa_block_sparse_attn(a, _dense(idx, "idx", (H, groups, n_sel), torch.int32, dev),
                                        n_sel, _int32(block, "block"), q_block, _stream(stream)), "ispa_block_sparse_attn")
    return {"o_loc": o_loc, "o_full": o_full, "d": d_out, "lse_loc": lse_loc, "lse_hist": lse_hist}


def select_layers(eps: Sequence[float], k: int):
    """ispa_select_layers (host): indices of the k lowest-eps layers (ascending index) and a 0/1 mask.
    Returns (idx int32 array, mask uint8 array, status)."""
    e = np.ascontiguousarray(np.asarray(eps, dtype=np.float64))
    n = int(e.shape[0])
    idx = np.zeros((max(k, 1),), dtype=np.int32)
    mask = np.zeros((max(n, 1),), dtype=np.uint8)
    st = lib().ispa_select_layers(e.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), n, int(k),
                                  idx.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                  mask.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8)))
    if st not in (ISPA_OK, ISPA_ERR_NONFINITE):
        raise IspaError(st, "ispa_select_layers")
    return idx[:k].copy(), mask[:n].copy(), st


def get_device_status(stream=None) -> int:
    return int(lib().ispa_get_device_status(_stream(stream)))


def test_set_flags(flags: int) -> None:
    """ispa_test_set_flags: process-wide test hooks (0 = off), for tests of the device-status path."""
    _check(lib().ispa_test_set_flags(int(flags)), "ispa_test_set_flags")


def launch_count() -> int:
    return int(lib().ispa_launch_count())


def version() -> int:
    return int(lib().ispa_version())

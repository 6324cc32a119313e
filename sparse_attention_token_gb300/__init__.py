"""Python binding of the GB300 DSA indexer library (libdsa_indexer.so).

Argument marshalling only: every step of the indexer runs in the CUDA kernels
behind the C ABI of include/dsa_indexer.h.  Tensors must be CUDA tensors; the
library is loaded with ctypes and there is no fallback -- if the library is
missing or a call fails, an exception is raised.

Function names mirror the C ABI:
  dsa_indexer_scores, dsa_indexer_topk, dsa_indexer, dsa_indexer_workspace_size,
  dsa_indexer_dense_host, dsa_indexer_dense_host_workspace_size, dsa_indexer_cache_append,
  dsa_resolve_indexer_sources, dsa_indexer_stack, dsa_check_device_status,
  dsa_topk_width, dsa_status_string, dsa_version (and the others the header declares;
  dsa_clock_sample is a diagnostic for measuring the SM clock over an interval).
Calls that take `stream` run on it (default: the current stream): what they allocate comes from
that stream's memory, and the caller orders the stream behind the kernels that made the inputs and
before those that read the results, as with torch's own operators under torch.cuda.stream(stream).
Host helpers from the GLM5 TensorCast adaptation design ("Sparse MLA 配置兼容",
"GLM-5.2 IndexShare"): resolve_topk_limit, extend_indexer_types_for_mtp,
indexer_types_to_codes.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdsa_indexer.so")

DSA_OK = 0
DSA_ERR_INVALID_ARGUMENT = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_CUDA = 3
DSA_ERR_DEVICE_CHECK = 4
DSA_ERR_TIMEOUT = 5
DSA_ERR_WORKSPACE = 6

DSA_BF16 = 0
DSA_FP8_E4M3 = 1
DSA_LAYER_FULL = 0
DSA_LAYER_SHARED = 1
DSA_ORDER_SCORE = 0
DSA_ORDER_INDEX = 1
DSA_MAX_TOPK = 4096


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dsa_status_string(status)} ({status})")


class dsa_indexer_args(ctypes.Structure):
    _fields_ = [
        ("q_dtype", ctypes.c_int), ("k_dtype", ctypes.c_int), ("B", ctypes.c_int),
        ("total_q", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("max_pages_per_seq", ctypes.c_int), ("max_seq_len", ctypes.c_int),
        ("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("w", ctypes.c_void_p),
        ("cu_q_lens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
        ("k_scale_cache", ctypes.c_void_p), ("topk_limit", ctypes.c_int), ("k_out", ctypes.c_int),
        ("order", ctypes.c_int), ("topk", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("k_new", ctypes.c_void_p), ("slot_mapping", ctypes.c_void_p),
    ]


class dsa_sparse_mla_args(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("total_q", ctypes.c_int), ("H", ctypes.c_int), ("kv_rank", ctypes.c_int),
                ("rope_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int), ("topk_width", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_nope", ctypes.c_void_p), ("q_rope", ctypes.c_void_p), ("cache_c", ctypes.c_void_p),
                ("cache_r", ctypes.c_void_p), ("block_tables", ctypes.c_void_p), ("cu_q_lens", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("topk", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class dsa_indexer_prepare_args(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int), ("hidden_dim", ctypes.c_int), ("q_rank", ctypes.c_int), ("H", ctypes.c_int),
        ("D", ctypes.c_int), ("rope_dim", ctypes.c_int), ("rope_interleaved", ctypes.c_int),
        ("hidden", ctypes.c_void_p), ("qa_normed", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
        ("rope_sin", ctypes.c_void_p), ("wq_b", ctypes.c_void_p), ("wk", ctypes.c_void_p),
        ("weights_proj", ctypes.c_void_p), ("k_norm_weight", ctypes.c_void_p), ("k_norm_bias", ctypes.c_void_p),
        ("k_norm_eps", ctypes.c_float), ("cache_dtype", ctypes.c_int), ("slot_mapping", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("k_scale_cache", ctypes.c_void_p), ("page_size", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("q_out", ctypes.c_void_p), ("q_scale_out", ctypes.c_void_p),
        ("w_out", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class dsa_page_plan_args(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("total_q", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int), ("num_prefix_pages", ctypes.c_int), ("num_free", ctypes.c_int),
                ("q_lens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("prefix_pages", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("block_tables", ctypes.c_void_p), ("cu_q_lens", ctypes.c_void_p),
                ("slot_mapping", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("used", ctypes.c_void_p)]


class dsa_mla_cache_append_args(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("kv_rank", ctypes.c_int), ("rope_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int), ("rope_interleaved", ctypes.c_int),
                ("rope_rows", ctypes.c_int), ("norm_eps", ctypes.c_float), ("c_kv", ctypes.c_void_p),
                ("k_rope", ctypes.c_void_p), ("c_stride", ctypes.c_int64), ("r_stride", ctypes.c_int64),
                ("slot_mapping", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
                ("rope_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("cache_c", ctypes.c_void_p),
                ("cache_r", ctypes.c_void_p)]


class dsa_prefix_mla_args(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("total_q", ctypes.c_int), ("H", ctypes.c_int), ("kv_rank", ctypes.c_int),
                ("rope_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int), ("prefix_len", ctypes.c_int), ("num_prefix_pages", ctypes.c_int),
                ("scale", ctypes.c_float), ("q_nope", ctypes.c_void_p), ("q_rope", ctypes.c_void_p),
                ("qn_stride_t", ctypes.c_int64), ("qn_stride_h", ctypes.c_int64), ("qr_stride_t", ctypes.c_int64),
                ("qr_stride_h", ctypes.c_int64), ("cache_c", ctypes.c_void_p), ("cache_r", ctypes.c_void_p),
                ("prefix_pages", ctypes.c_void_p), ("block_tables", ctypes.c_void_p), ("cu_q_lens", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_LIB = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.dsa_status_string.restype = ctypes.c_char_p
        L.dsa_status_string.argtypes = [I]
        L.dsa_version.restype = ctypes.c_char_p
        L.dsa_topk_width.restype = I
        L.dsa_topk_width.argtypes = [I, I64]
        L.dsa_indexer_scores.restype = I
        L.dsa_indexer_scores.argtypes = [P, I, P, P, I, P, P, I, I, I, I, I, P, I64, P]
        L.dsa_indexer_topk.restype = I
        L.dsa_indexer_topk.argtypes = [P, I64, I, I, I, I, I, I, P, P]
        L.dsa_indexer_workspace_size.restype = I
        L.dsa_indexer_workspace_size.argtypes = [ctypes.POINTER(dsa_indexer_args), ctypes.POINTER(S)]
        L.dsa_indexer.restype = I
        L.dsa_indexer.argtypes = [ctypes.POINTER(dsa_indexer_args), P]
        L.dsa_resolve_indexer_sources.restype = I
        L.dsa_resolve_indexer_sources.argtypes = [I, P, P]
        L.dsa_indexer_stack.restype = I
        L.dsa_indexer_stack.argtypes = [I, P, P, P, P, P]
        L.dsa_check_device_status.restype = I
        L.dsa_check_device_status.argtypes = [P]
        L.dsa_clock_sample.restype = I
        L.dsa_clock_sample.argtypes = [P, I, P]
        L.dsa_indexer_prepare_workspace_size.restype = I
        L.dsa_indexer_prepare_workspace_size.argtypes = [ctypes.POINTER(dsa_indexer_prepare_args), ctypes.POINTER(S)]
        L.dsa_indexer_prepare.restype = I
        L.dsa_indexer_prepare.argtypes = [ctypes.POINTER(dsa_indexer_prepare_args), P]
        L.dsa_indexer_cache_append.restype = I
        L.dsa_indexer_cache_append.argtypes = [P, I, I, P, P, I, P, I, I, P]
        L.dsa_indexer_dense_host_workspace_size.restype = I
        L.dsa_indexer_dense_host_workspace_size.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(S)]
        L.dsa_indexer_dense_host.restype = I
        L.dsa_indexer_dense_host.argtypes = [P, I, P, P, I, P, P, I, I, I, I, I, I, I, I, I, P, P, S, P]
        L.dsa_indexer_shard_candidates_workspace_size.restype = I
        L.dsa_indexer_shard_candidates_workspace_size.argtypes = [I, I, ctypes.POINTER(S)]
        L.dsa_indexer_shard_candidates.restype = I
        L.dsa_indexer_shard_candidates.argtypes = [P, I, P, P, I, P, P, I, I, I, I, I, I, I, P, P, P, S, P]
        L.dsa_indexer_merge_candidates.restype = I
        L.dsa_indexer_merge_candidates.argtypes = [P, P, I, I, I, I, I, I, P, P]
        L.dsa_sparse_mla_workspace_size.restype = I
        L.dsa_sparse_mla_workspace_size.argtypes = [ctypes.POINTER(dsa_sparse_mla_args), ctypes.POINTER(S)]
        L.dsa_sparse_mla.restype = I
        L.dsa_sparse_mla.argtypes = [ctypes.POINTER(dsa_sparse_mla_args), P]
        L.dsa_page_plan.restype = I
        L.dsa_page_plan.argtypes = [P, P]
        L.dsa_mla_cache_append.restype = I
        L.dsa_mla_cache_append.argtypes = [P, P]
        L.dsa_prefix_mla_workspace_size.restype = I
        L.dsa_prefix_mla_workspace_size.argtypes = [P, ctypes.POINTER(S)]
        L.dsa_prefix_mla.restype = I
        L.dsa_prefix_mla.argtypes = [P, P]
        L.dsa_test_arm_score_timeout.restype = I
        L.dsa_test_arm_score_timeout.argtypes = [ctypes.c_ulonglong]
        L.dsa_test_arm_prefix_mla_timeout.restype = I
        L.dsa_test_arm_prefix_mla_timeout.argtypes = [I, ctypes.c_uint, ctypes.c_ulonglong]
        _LIB = L
    return _LIB


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DsaError(status, where)


def dsa_status_string(status: int) -> str:
    return lib().dsa_status_string(int(status)).decode()


def dsa_version() -> str:
    return lib().dsa_version().decode()


def dsa_topk_width(topk_limit: int, active_seq_len: int) -> int:
    return int(lib().dsa_topk_width(int(topk_limit), int(active_seq_len)))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    if t.dtype == torch.float8_e4m3fn:
        return DSA_FP8_E4M3
    raise TypeError(f"unsupported element type {t.dtype} (bf16 or float8_e4m3fn)")


def _on_current_device(t: torch.Tensor, name: str) -> None:
    """The library launches on the calling thread's current device, so every tensor lies there."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    here = torch._C._cuda_getDevice()
    if t.get_device() != here:
        raise ValueError(f"{name} is on cuda:{t.get_device()} but the current device is cuda:{here}: call under "
                         f"torch.cuda.device({t.get_device()})")


def _dev(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    _on_current_device(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    """Raw cudaStream_t of `stream` (default: torch's current stream; NULL without CUDA)."""
    if stream is None:
        if not torch.cuda.is_available():
            return None
        stream = torch.cuda.current_stream()
    elif stream.device_index != torch._C._cuda_getDevice():
        raise ValueError(f"stream is one of cuda:{stream.device_index} but the current device is "
                         f"cuda:{torch._C._cuda_getDevice()}")
    return stream.cuda_stream


def _on(stream):
    """Where a call allocates: on the stream that its kernels run on.  A block of another stream's
    memory may still be in use by kernels queued there, which nothing orders before this call's."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _hold(stream, inputs, results=()) -> None:
    """After a call on a given stream: the caller may drop its tensors, and use and drop the
    results on its current stream, without their memory being reused ahead of either's kernels
    (the allocator itself only knows the stream that a tensor was allocated on)."""
    if stream is None:
        return
    here = torch.cuda.current_stream()
    if here == stream:
        return
    for tensors, on in ((inputs, stream), (results, here)):
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(on)


def _expect(checks) -> None:
    """Raise ValueError unless every (tensor or None, name, shape) matches; a shape entry
    of None accepts any size in that dimension.  The C ABI sees only pointers and sizes."""
    for t, name, shape in checks:
        if t is None:
            continue
        ok = t.dim() == len(shape) and all(w is None or t.shape[i] == w for i, w in enumerate(shape))
        if not ok:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def dsa_indexer_scores(q: torch.Tensor, k: torch.Tensor, w: torch.Tensor, *, q_pos0: Optional[int] = None,
                       q_scale: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                       scores: Optional[torch.Tensor] = None, ld: Optional[int] = None,
                       fill=float("-inf"), stream=None) -> torch.Tensor:
    """Dense scores [T, ld] fp32 of queries q [T, H, D] against keys k [S, D].

    Entries a query cannot see (s > q_pos0 + t) are left as the output buffer held
    them: a freshly allocated buffer is filled with ``fill`` (by torch) first."""
    T, H, D = q.shape
    S = k.shape[0]
    if q_pos0 is None:
        q_pos0 = S - T
    if ld is None:
        ld = (S + 3) // 4 * 4
    if scores is None:
        with _on(stream):
            scores = torch.full((T, ld), fill, dtype=torch.float32, device=q.device)
    _expect([(k, "k", (S, D)), (w, "w", (T, H)), (q_scale, "q_scale", (T, H)), (k_scale, "k_scale", (S,)),
             (scores, "scores", (T, None))])
    if scores.shape[1] < S:
        raise ValueError(f"scores needs at least S = {S} columns, got {scores.shape[1]}")
    _check(lib().dsa_indexer_scores(
        _dev(q, "q"), _dtype_code(q), _dev(q_scale, "q_scale", torch.float32),
        _dev(k, "k"), _dtype_code(k), _dev(k_scale, "k_scale", torch.float32),
        _dev(w, "w", torch.float32), T, S, H, D, int(q_pos0), _dev(scores, "scores", torch.float32),
        int(scores.stride(0)), _stream_ptr(stream)), "dsa_indexer_scores")
    _hold(stream, (q, k, w, q_scale, k_scale, scores), (scores,))
    return scores


def _host(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def dsa_indexer_dense_host_workspace_size(T: int, S: int, H: int, D: int, q_dtype: int, k_out: int,
                                          chunk_rows: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().dsa_indexer_dense_host_workspace_size(T, S, H, D, q_dtype, k_out, chunk_rows, ctypes.byref(n)),
           "dsa_indexer_dense_host_workspace_size")
    return int(n.value)


def dsa_indexer_dense_host(q: torch.Tensor, k: torch.Tensor, w: torch.Tensor, *, topk_limit: int,
                           q_pos0: Optional[int] = None, k_out: Optional[int] = None, order: int = DSA_ORDER_SCORE,
                           q_scale: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                           chunk_rows: int = 0, topk: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scores + top-k of one sequence from HOST tensors q [T, H, D], k [S, D], w [T, H]
    (pin them for overlapped copies) into a host int32 [T, k_out] tensor; the transfers
    are chunked and overlapped with the kernels.  `workspace`: a CUDA uint8 tensor of at
    least dsa_indexer_dense_host_workspace_size bytes (allocated when omitted).  The
    result is final once `stream` (default: torch's current stream) is synchronised."""
    T, H, D = q.shape
    S = k.shape[0]
    if q_pos0 is None:
        q_pos0 = S - T
    if k_out is None:
        k_out = topk_limit
    if topk is None:
        topk = torch.empty((T, k_out), dtype=torch.int32, pin_memory=torch.cuda.is_available())
    _expect([(k, "k", (S, D)), (w, "w", (T, H)), (q_scale, "q_scale", (T, H)), (k_scale, "k_scale", (S,)),
             (topk, "topk", (T, k_out))])
    need = dsa_indexer_dense_host_workspace_size(T, S, H, D, _dtype_code(q), k_out, chunk_rows)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    if not workspace.is_cuda or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a CUDA uint8 tensor")
    _on_current_device(workspace, "workspace")
    _check(lib().dsa_indexer_dense_host(
        _host(q, "q"), _dtype_code(q), _host(q_scale, "q_scale", torch.float32),
        _host(k, "k"), _dtype_code(k), _host(k_scale, "k_scale", torch.float32),
        _host(w, "w", torch.float32), T, S, H, D, int(q_pos0), int(topk_limit), int(k_out), int(order),
        int(chunk_rows), _host(topk, "topk", torch.int32), workspace.data_ptr(), workspace.numel(),
        _stream_ptr(stream)), "dsa_indexer_dense_host")
    _hold(stream, (workspace,))
    return topk


def dsa_indexer_topk(scores: torch.Tensor, *, T: int, S: int, q_pos0: int, topk_limit: int,
                     k_out: Optional[int] = None, order: int = DSA_ORDER_SCORE,
                     topk: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-row top-k [T, k_out] int32 of dense scores (row t sees min(q_pos0 + t + 1, S) keys)."""
    if k_out is None:
        k_out = topk_limit
    if topk is None:
        with _on(stream):
            topk = torch.empty((T, k_out), dtype=torch.int32, device=scores.device)
    _expect([(scores, "scores", (None, None)), (topk, "topk", (T, k_out))])
    if scores.shape[0] < T or scores.shape[1] < S:
        raise ValueError(f"scores must hold at least [{T}, {S}], got {tuple(scores.shape)}")
    _check(lib().dsa_indexer_topk(_dev(scores, "scores", torch.float32), int(scores.stride(0)), T, S,
                                  int(q_pos0), int(topk_limit), int(k_out), int(order),
                                  _dev(topk, "topk", torch.int32), _stream_ptr(stream)), "dsa_indexer_topk")
    _hold(stream, (scores, topk), (topk,))
    return topk


def make_indexer_args(q, w, k_cache, cu_q_lens, seq_lens, block_tables, *, max_seq_len: int, topk_limit: int,
                      k_out: Optional[int] = None, q_scale=None, k_scale_cache=None, topk=None,
                      workspace=None, order: int = DSA_ORDER_SCORE, total_q: Optional[int] = None,
                      k_new=None, slot_mapping=None):
    """Fill a dsa_indexer_args from tensors (allocating topk / workspace with torch if absent).

    Returns (args, keepalive) -- keep the second value alive while the call runs."""
    if q.dim() != 3 or k_cache.dim() != 3 or seq_lens.dim() != 1 or block_tables.dim() != 2:
        raise ValueError("q [total_q, H, D], k_cache [num_pages, page_size, D], seq_lens [B] and "
                         "block_tables [B, max_pages] expected")
    total_q = q.shape[0] if total_q is None else total_q
    H, D = q.shape[1], q.shape[2]
    B = seq_lens.shape[0]
    num_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    if k_out is None:
        k_out = topk_limit
    if topk is None:
        topk = torch.empty((total_q, k_out), dtype=torch.int32, device=q.device)
    # the C ABI sees only pointers and sizes: every tensor's shape is checked here
    want = {"w": (w, (q.shape[0], H)), "q_scale": (q_scale, (q.shape[0], H)),
            "k_scale_cache": (k_scale_cache, (num_pages, page_size)), "cu_q_lens": (cu_q_lens, (B + 1,)),
            "block_tables": (block_tables, (B, block_tables.shape[1])), "topk": (topk, (total_q, k_out)),
            "k_new": (k_new, (total_q, D)), "slot_mapping": (slot_mapping, (total_q,))}
    for name, (t, shape) in want.items():
        if t is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if k_cache.shape[2] != D or q.shape[0] < total_q:
        raise ValueError(f"k_cache rows must have D = {D} values and q at least {total_q} rows")
    a = dsa_indexer_args()
    a.q_dtype, a.k_dtype = _dtype_code(q), _dtype_code(k_cache)
    a.B, a.total_q, a.H, a.D = B, total_q, H, D
    a.page_size, a.num_pages = page_size, num_pages
    a.max_pages_per_seq, a.max_seq_len = block_tables.shape[1], int(max_seq_len)
    a.q = _dev(q, "q")
    a.q_scale = _dev(q_scale, "q_scale", torch.float32)
    a.w = _dev(w, "w", torch.float32)
    a.cu_q_lens = _dev(cu_q_lens, "cu_q_lens", torch.int32)
    a.seq_lens = _dev(seq_lens, "seq_lens", torch.int32)
    a.block_tables = _dev(block_tables, "block_tables", torch.int32)
    a.k_cache = _dev(k_cache, "k_cache")
    a.k_scale_cache = _dev(k_scale_cache, "k_scale_cache", torch.float32)
    a.topk_limit, a.k_out, a.order = int(topk_limit), int(k_out), int(order)
    a.topk = _dev(topk, "topk", torch.int32)
    if workspace is None:
        nbytes = dsa_indexer_workspace_size(a)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    a.workspace = _dev(workspace, "workspace", torch.uint8)
    a.workspace_bytes = workspace.numel()
    if (k_new is None) != (slot_mapping is None):
        raise ValueError("k_new and slot_mapping go together")
    a.k_new = _dev(k_new, "k_new", torch.bfloat16)
    a.slot_mapping = _dev(slot_mapping, "slot_mapping", torch.int64)
    return a, (q, w, k_cache, cu_q_lens, seq_lens, block_tables, q_scale, k_scale_cache, topk, workspace, k_new,
               slot_mapping)


def dsa_indexer_workspace_size(args: dsa_indexer_args) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().dsa_indexer_workspace_size(ctypes.byref(args), ctypes.byref(n)), "dsa_indexer_workspace_size")
    return int(n.value)


def dsa_indexer(q, w, k_cache, cu_q_lens, seq_lens, block_tables, *, max_seq_len: int, topk_limit: int,
                k_out: Optional[int] = None, q_scale=None, k_scale_cache=None, topk=None, workspace=None,
                order: int = DSA_ORDER_SCORE, k_new=None, slot_mapping=None, stream=None) -> torch.Tensor:
    """Fused paged indexer for a varlen batch; returns topk [total_q, k_out] int32.
    With k_new [total_q, D] bf16 and slot_mapping [total_q] int64 the step's keys are
    first written into k_cache (and k_scale_cache), in place."""
    with _on(stream):
        a, keep = make_indexer_args(q, w, k_cache, cu_q_lens, seq_lens, block_tables, max_seq_len=max_seq_len,
                                    topk_limit=topk_limit, k_out=k_out, q_scale=q_scale,
                                    k_scale_cache=k_scale_cache, topk=topk, workspace=workspace, order=order,
                                    k_new=k_new, slot_mapping=slot_mapping)
    _check(lib().dsa_indexer(ctypes.byref(a), _stream_ptr(stream)), "dsa_indexer")
    _hold(stream, keep, (keep[8],))
    return keep[8]


def dsa_indexer_cache_append(k_new: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                             k_scale_cache: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write new bf16 key rows k_new [n, D] into k_cache [num_pages, page_size, D] at the
    slots slot_mapping [n] (int64, page * page_size + row; negative = skip), in place;
    an e4m3 cache takes them quantised with one scale amax/448 per token into
    k_scale_cache [num_pages, page_size]."""
    n, D = k_new.shape
    num_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    _expect([(slot_mapping, "slot_mapping", (n,)), (k_cache, "k_cache", (None, None, D)),
             (k_scale_cache, "k_scale_cache", (num_pages, page_size))])
    _check(lib().dsa_indexer_cache_append(
        _dev(k_new, "k_new", torch.bfloat16), n, D, _dev(slot_mapping, "slot_mapping", torch.int64),
        _dev(k_cache, "k_cache"), _dtype_code(k_cache), _dev(k_scale_cache, "k_scale_cache", torch.float32),
        page_size, num_pages, _stream_ptr(stream)), "dsa_indexer_cache_append")
    _hold(stream, (k_new, slot_mapping, k_cache, k_scale_cache))


def make_prepare_args(hidden: torch.Tensor, qa_normed: torch.Tensor, rope_cos: Optional[torch.Tensor],
                      rope_sin: Optional[torch.Tensor], wq_b: torch.Tensor, wk: torch.Tensor,
                      weights_proj: torch.Tensor, k_norm_weight: torch.Tensor, k_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, *, H: int, rope_dim: int, rope_interleaved: bool = False,
                      k_norm_bias: Optional[torch.Tensor] = None, k_norm_eps: float = 1e-6,
                      k_scale_cache: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """(args, keepalive, (q, q_scale, w)) for dsa_indexer_prepare: allocates the outputs
    (q [T, H, D] in the cache's element type, q_scale [T, H] for an e4m3 cache, w [T, H])
    and, unless given, the workspace."""
    T, hidden_dim = hidden.shape
    q_rank = qa_normed.shape[1]
    D = wk.shape[0]
    fp8 = k_cache.dtype == torch.float8_e4m3fn
    # the C ABI sees only pointers and sizes: every tensor's shape is checked here
    want = {"qa_normed": (qa_normed, (T, q_rank)), "wq_b": (wq_b, (H * D, q_rank)), "wk": (wk, (D, hidden_dim)),
            "weights_proj": (weights_proj, (H, hidden_dim)), "k_norm_weight": (k_norm_weight, (D,)),
            "slot_mapping": (slot_mapping, (T,))}
    if k_norm_bias is not None:
        want["k_norm_bias"] = (k_norm_bias, (D,))
    if rope_dim > 0:
        want["rope_cos"] = (rope_cos, (T, rope_dim // 2))
        want["rope_sin"] = (rope_sin, (T, rope_dim // 2))
    if k_cache.dim() != 3 or k_cache.shape[2] != D:
        raise ValueError(f"k_cache must be [num_pages, page_size, {D}], got {tuple(k_cache.shape)}")
    if fp8:
        want["k_scale_cache"] = (k_scale_cache, tuple(k_cache.shape[:2]))
    for name, (t, shape) in want.items():
        if t is None or tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {None if t is None else tuple(t.shape)}")
    dev = hidden.device
    q = torch.empty((T, H, D), dtype=k_cache.dtype, device=dev)
    q_scale = torch.empty((T, H), dtype=torch.float32, device=dev) if fp8 else None
    w = torch.empty((T, H), dtype=torch.float32, device=dev)
    a = dsa_indexer_prepare_args()
    a.T, a.hidden_dim, a.q_rank, a.H, a.D = T, hidden_dim, q_rank, H, D
    a.rope_dim, a.rope_interleaved = rope_dim, 1 if rope_interleaved else 0
    a.hidden = _dev(hidden, "hidden", torch.bfloat16)
    a.qa_normed = _dev(qa_normed, "qa_normed", torch.bfloat16)
    a.rope_cos = _dev(rope_cos, "rope_cos", torch.float32)
    a.rope_sin = _dev(rope_sin, "rope_sin", torch.float32)
    a.wq_b = _dev(wq_b, "wq_b", torch.bfloat16)
    a.wk = _dev(wk, "wk", torch.bfloat16)
    a.weights_proj = _dev(weights_proj, "weights_proj", torch.bfloat16)
    a.k_norm_weight = _dev(k_norm_weight, "k_norm_weight", torch.float32)
    a.k_norm_bias = _dev(k_norm_bias, "k_norm_bias", torch.float32)
    a.k_norm_eps = float(k_norm_eps)
    a.cache_dtype = _dtype_code(k_cache)
    a.slot_mapping = _dev(slot_mapping, "slot_mapping", torch.int64)
    a.k_cache = _dev(k_cache, "k_cache")
    a.k_scale_cache = _dev(k_scale_cache, "k_scale_cache", torch.float32)
    a.page_size, a.num_pages = k_cache.shape[1], k_cache.shape[0]
    a.q_out, a.q_scale_out, a.w_out = q.data_ptr(), _dev(q_scale, "q_scale"), w.data_ptr()
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(lib().dsa_indexer_prepare_workspace_size(ctypes.byref(a), ctypes.byref(n)),
               "dsa_indexer_prepare_workspace_size")
        workspace = torch.empty(max(int(n.value), 1), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    keep = [hidden, qa_normed, rope_cos, rope_sin, wq_b, wk, weights_proj, k_norm_weight, k_norm_bias, k_cache,
            slot_mapping, k_scale_cache, q, q_scale, w, workspace]
    return a, keep, (q, q_scale, w)


def dsa_indexer_prepare(hidden: torch.Tensor, qa_normed: torch.Tensor, rope_cos: Optional[torch.Tensor],
                        rope_sin: Optional[torch.Tensor], wq_b: torch.Tensor, wk: torch.Tensor,
                        weights_proj: torch.Tensor, k_norm_weight: torch.Tensor, k_cache: torch.Tensor,
                        slot_mapping: torch.Tensor, *, H: int, rope_dim: int, rope_interleaved: bool = False,
                        k_norm_bias: Optional[torch.Tensor] = None, k_norm_eps: float = 1e-6,
                        k_scale_cache: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None):
    """The indexer front-end through the C ABI: returns (q, q_scale, w) for dsa_indexer
    and writes this step's keys (and on an e4m3 cache their scales) through slot_mapping."""
    with _on(stream):
        a, keep, out = make_prepare_args(
            hidden, qa_normed, rope_cos, rope_sin, wq_b, wk, weights_proj, k_norm_weight, k_cache, slot_mapping, H=H,
            rope_dim=rope_dim, rope_interleaved=rope_interleaved, k_norm_bias=k_norm_bias, k_norm_eps=k_norm_eps,
            k_scale_cache=k_scale_cache, workspace=workspace)
    _check(lib().dsa_indexer_prepare(ctypes.byref(a), _stream_ptr(stream)), "dsa_indexer_prepare")
    _hold(stream, keep, out)
    return out


def indexer_types_to_codes(indexer_types: Sequence) -> list:
    """'full' / 'shared' (or the integer codes) -> dsa_layer_type codes; others -> -1."""
    out = []
    for t in indexer_types:
        if t in ("full", DSA_LAYER_FULL):
            out.append(DSA_LAYER_FULL)
        elif t in ("shared", DSA_LAYER_SHARED):
            out.append(DSA_LAYER_SHARED)
        else:
            out.append(-1)
    return out


def dsa_resolve_indexer_sources(indexer_types: Sequence, num_layers: Optional[int] = None) -> list:
    """Source layer of every layer through the C ABI; ValueError like the reference flow
    for a short list, an unknown type or a shared layer with no earlier full layer."""
    codes = indexer_types_to_codes(indexer_types)
    if num_layers is not None and len(codes) < num_layers:
        raise ValueError("indexer_types shorter than the number of layers")
    L = len(codes)
    types = (ctypes.c_int32 * max(L, 1))(*codes)
    src = (ctypes.c_int32 * max(L, 1))()
    st = lib().dsa_resolve_indexer_sources(L, ctypes.cast(types, ctypes.c_void_p), ctypes.cast(src, ctypes.c_void_p))
    if st == DSA_ERR_INVALID_ARGUMENT:
        raise ValueError("invalid indexer_types: unknown type or shared layer without an earlier full layer")
    _check(st, "dsa_resolve_indexer_sources")
    return list(src[:L])


def dsa_indexer_stack(indexer_types: Sequence, full_layer_args: Sequence, stream=None):
    """Run an IndexShare stack.  full_layer_args[l] is a dsa_indexer_args (full layers)
    or None (shared layers).  Returns (topk device pointers per layer, source layers)."""
    codes = indexer_types_to_codes(indexer_types)
    L = len(codes)
    types = (ctypes.c_int32 * max(L, 1))(*codes)
    arr = (ctypes.POINTER(dsa_indexer_args) * max(L, 1))()
    for i, a in enumerate(full_layer_args):
        arr[i] = ctypes.pointer(a) if a is not None else ctypes.POINTER(dsa_indexer_args)()
    outs = (ctypes.c_void_p * max(L, 1))()
    src = (ctypes.c_int32 * max(L, 1))()
    st = lib().dsa_indexer_stack(L, ctypes.cast(types, ctypes.c_void_p), ctypes.cast(arr, ctypes.c_void_p),
                                 ctypes.cast(outs, ctypes.c_void_p), ctypes.cast(src, ctypes.c_void_p),
                                 _stream_ptr(stream))
    _check(st, "dsa_indexer_stack")
    return [outs[i] for i in range(L)], list(src[:L])


# ---- key-sharded top-k (GLM5 LoRA blog, section 3.1: context parallelism) ---------------

def dsa_indexer_shard_candidates(q: torch.Tensor, k_shard: torch.Tensor, w: torch.Tensor, *, q_pos0: int,
                                 key_offset: int, k_cand: int, q_scale: Optional[torch.Tensor] = None,
                                 k_scale: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                 stream=None):
    """One key shard's candidates: (cand_idx [T, k_cand] int32 global indices then -1,
    cand_scores [T, k_cand] fp32 then -inf) for keys key_offset .. key_offset + S - 1."""
    T, H, D = q.shape
    S = k_shard.shape[0]
    _expect([(k_shard, "k_shard", (S, D)), (w, "w", (T, H)), (q_scale, "q_scale", (T, H)),
             (k_scale, "k_scale", (S,))])
    nbytes = ctypes.c_size_t(0)
    _check(lib().dsa_indexer_shard_candidates_workspace_size(T, S, ctypes.byref(nbytes)),
           "dsa_indexer_shard_candidates_workspace_size")
    with _on(stream):
        if workspace is None:
            workspace = torch.empty(max(nbytes.value, 16), dtype=torch.uint8, device=q.device)
        cand_idx = torch.empty((T, k_cand), dtype=torch.int32, device=q.device)
        cand_scores = torch.empty((T, k_cand), dtype=torch.float32, device=q.device)
    _check(lib().dsa_indexer_shard_candidates(
        _dev(q, "q"), _dtype_code(q), _dev(q_scale, "q_scale", torch.float32), _dev(k_shard, "k_shard"),
        _dtype_code(k_shard), _dev(k_scale, "k_scale", torch.float32), _dev(w, "w", torch.float32), T, S, H, D,
        int(q_pos0), int(key_offset), int(k_cand), cand_idx.data_ptr(), cand_scores.data_ptr(),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
        "dsa_indexer_shard_candidates")
    _hold(stream, (q, k_shard, w, q_scale, k_scale, workspace), (cand_idx, cand_scores))
    return cand_idx, cand_scores


def dsa_indexer_merge_candidates(cand_scores: torch.Tensor, cand_idx: torch.Tensor, *, topk_limit: int,
                                 k_out: Optional[int] = None, order: int = DSA_ORDER_SCORE,
                                 topk: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Top-k [T, k_out] of the union of the shards' candidates [n_shards, T, k_cand]."""
    n_shards, T, k_cand = cand_idx.shape
    k_out = topk_limit if k_out is None else k_out
    _expect([(cand_scores, "cand_scores", (n_shards, T, k_cand))])
    if topk is None:
        with _on(stream):
            topk = torch.empty((T, k_out), dtype=torch.int32, device=cand_idx.device)
    _expect([(topk, "topk", (T, k_out))])
    _check(lib().dsa_indexer_merge_candidates(
        _dev(cand_scores, "cand_scores", torch.float32), _dev(cand_idx, "cand_idx", torch.int32), n_shards, T,
        k_cand, int(topk_limit), int(k_out), int(order), _dev(topk, "topk", torch.int32), _stream_ptr(stream)),
        "dsa_indexer_merge_candidates")
    _hold(stream, (cand_scores, cand_idx, topk), (topk,))
    return topk


def gather_shard_candidates(cand_idx: torch.Tensor, cand_scores: torch.Tensor, group=None):
    """The candidates of every rank of `group`, stacked in rank order: ([world, T, k] int32,
    [world, T, k] fp32).  One all-gather of indices and one of scores (torch.distributed;
    NCCL for device tensors, gloo for host tensors)."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    idx = [torch.empty_like(cand_idx) for _ in range(world)]
    sc = [torch.empty_like(cand_scores) for _ in range(world)]
    dist.all_gather(idx, cand_idx.contiguous(), group=group)
    dist.all_gather(sc, cand_scores.contiguous(), group=group)
    return torch.stack(idx), torch.stack(sc)


def dsa_indexer_key_sharded(q: torch.Tensor, k_shard: torch.Tensor, w: torch.Tensor, *, q_pos0: int,
                            key_offset: int, topk_limit: int, k_out: Optional[int] = None,
                            order: int = DSA_ORDER_SCORE, q_scale: Optional[torch.Tensor] = None,
                            k_scale: Optional[torch.Tensor] = None, group=None, stream=None) -> torch.Tensor:
    """Top-k over a sequence whose keys are split over the ranks of `group` (each rank holds
    the queries and its own contiguous key shard): local candidates, one all-gather, merge."""
    k_out = topk_limit if k_out is None else k_out
    ci, cs = dsa_indexer_shard_candidates(q, k_shard, w, q_pos0=q_pos0, key_offset=key_offset,
                                          k_cand=min(topk_limit, k_out), q_scale=q_scale, k_scale=k_scale,
                                          stream=stream)
    with _on(stream):  # the gather reads what the call above writes on that stream
        all_idx, all_sc = gather_shard_candidates(ci, cs, group)
    return dsa_indexer_merge_candidates(all_sc, all_idx, topk_limit=topk_limit, k_out=k_out, order=order,
                                        stream=stream)


# ---- sparse MLA over the top-k (the attention that consumes topk_indices) -----------------

def make_sparse_mla_args(q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, topk, *,
                         scale: float, out=None, workspace=None):
    """dsa_sparse_mla_args for these tensors (every shape checked); returns (args, kept tensors)."""
    total_q, H, R = q_nope.shape
    rd = q_rope.shape[2]
    num_pages, page_size = cache_c.shape[0], cache_c.shape[1]
    B = seq_lens.shape[0]
    k = topk.shape[1]
    _expect([(q_rope, "q_rope", (total_q, H, rd)), (cache_c, "cache_c", (num_pages, page_size, R)),
             (cache_r, "cache_r", (num_pages, page_size, rd)), (cu_q_lens, "cu_q_lens", (B + 1,)),
             (block_tables, "block_tables", (B, None)), (topk, "topk", (total_q, k))])
    if out is None:
        out = torch.empty((total_q, H, R), dtype=torch.float32, device=q_nope.device)
    _expect([(out, "out", (total_q, H, R))])
    a = dsa_sparse_mla_args()
    a.B, a.total_q, a.H, a.kv_rank, a.rope_dim = B, total_q, H, R, rd
    a.page_size, a.num_pages, a.max_pages_per_seq, a.topk_width = page_size, num_pages, block_tables.shape[1], k
    a.scale = float(scale)
    a.q_nope, a.q_rope = _dev(q_nope, "q_nope", torch.bfloat16), _dev(q_rope, "q_rope", torch.bfloat16)
    a.cache_c, a.cache_r = _dev(cache_c, "cache_c", torch.bfloat16), _dev(cache_r, "cache_r", torch.bfloat16)
    a.block_tables = _dev(block_tables, "block_tables", torch.int32)
    a.cu_q_lens = _dev(cu_q_lens, "cu_q_lens", torch.int32)
    a.seq_lens = _dev(seq_lens, "seq_lens", torch.int32)
    a.topk = _dev(topk, "topk", torch.int32)
    a.out = _dev(out, "out", torch.float32)
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(lib().dsa_sparse_mla_workspace_size(ctypes.byref(a), ctypes.byref(n)), "dsa_sparse_mla_workspace_size")
        workspace = torch.empty(max(n.value, 16), dtype=torch.uint8, device=q_nope.device)
    a.workspace = _dev(workspace, "workspace")
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a, (q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, topk, out, workspace)


def dsa_sparse_mla(q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, topk, *, scale: float,
                   out=None, workspace=None, stream=None) -> torch.Tensor:
    """Latent attention output [total_q, H, kv_rank] fp32 of each query over its selected keys."""
    with _on(stream):
        a, keep = make_sparse_mla_args(q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, topk,
                                       scale=scale, out=out, workspace=workspace)
    _check(lib().dsa_sparse_mla(ctypes.byref(a), _stream_ptr(stream)), "dsa_sparse_mla")
    _hold(stream, keep, (keep[8],))
    return keep[8]


# ---- a batch that shares its prompt: page plan, latent cache append, attention --------------

# These calls are often short against what it takes to make them, so their arguments are packed
# with struct (in the layout of the C structs above) and every check is one comparison that
# succeeds; the messages are put together only when one fails.
_PLAN_ARGS = struct.Struct("@6i9P")
_APPEND_ARGS = struct.Struct("@7if2P2q7P")
_PREFIX_ARGS = struct.Struct("@10if2P4q9PN")
assert _PLAN_ARGS.size == ctypes.sizeof(dsa_page_plan_args)
assert _APPEND_ARGS.size == ctypes.sizeof(dsa_mla_cache_append_args)
assert _PREFIX_ARGS.size == ctypes.sizeof(dsa_prefix_mla_args)


def _here(t: torch.Tensor) -> int:
    """Index of the current device, which every tensor of a call must lie on (no index where t,
    one of them, is no CUDA tensor: there may be no device to ask for)."""
    return torch._C._cuda_getDevice() if t.is_cuda else -2


def _ptr(t: Optional[torch.Tensor], name: str, dtype, here: int) -> int:
    """Device pointer of a contiguous tensor of this type on device `here` (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.get_device() != here or not t.is_contiguous():
        _dev(t, name, dtype)
    return t.data_ptr()


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor for the call's kernels, from the memory of the stream they run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, device, here, stream) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    if t.shape != shape:
        _expect([(t, name, shape)])
    _ptr(t, name, dtype, here)
    return t


def _rows(t: torch.Tensor, name: str, here: int) -> int:
    """Device pointer of a bf16 tensor on device `here` whose last dimension is dense, the others
    in any strides."""
    if t.get_device() != here:
        _on_current_device(t, name)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return t.data_ptr()


def _stream_of(here: int, stream) -> int:
    """Raw cudaStream_t of `stream`, or of the current stream on device `here`."""
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else _stream_ptr(stream)


def dsa_page_plan(q_lens: torch.Tensor, seq_lens: torch.Tensor, block_tables: torch.Tensor, free_pages: torch.Tensor,
                  *, page_size: int, total_q: int, prefix_pages: Optional[torch.Tensor] = None, cu_q_lens=None,
                  slot_mapping=None, positions=None, used=None, stream=None):
    """Block tables, slots, positions and query offsets of a step from the request lengths.

    Request b holds seq_lens[b] tokens after the step, the last q_lens[b] of them new.
    block_tables [B, max_pages] is updated in place: the shared prompt's whole pages
    (prefix_pages) in front, the pages a request already holds kept, new ones from the front
    of free_pages in request order, -1 behind.  total_q: the outputs' length, at least the
    sum of q_lens (the rest is -1).  Returns (cu_q_lens [B + 1] int32, slot_mapping [total_q]
    int64, positions [total_q] int32, used [1] int32: the free pages taken)."""
    bs, qs, fs = block_tables.shape, q_lens.shape, free_pages.shape
    n_prefix = 0 if prefix_pages is None else prefix_pages.shape[0] if prefix_pages.dim() == 1 else -1
    if len(qs) != 1 or len(bs) != 2 or len(fs) != 1 or n_prefix < 0 or bs[0] != qs[0] or seq_lens.shape != qs:
        B = qs[0] if len(qs) == 1 else None
        _expect([(q_lens, "q_lens", (None,)), (seq_lens, "seq_lens", (B,)), (block_tables, "block_tables", (B, None)),
                 (free_pages, "free_pages", (None,)), (prefix_pages, "prefix_pages", (None,))])
    B, width = bs
    i32, dev, here = torch.int32, block_tables.device, _here(block_tables)
    lens = (_ptr(q_lens, "q_lens", i32, here), _ptr(seq_lens, "seq_lens", i32, here),
            _ptr(prefix_pages, "prefix_pages", i32, here), _ptr(free_pages, "free_pages", i32, here),
            _ptr(block_tables, "block_tables", i32, here))
    cu_q_lens = _out(cu_q_lens, "cu_q_lens", (B + 1,), i32, dev, here, stream)
    slot_mapping = _out(slot_mapping, "slot_mapping", (total_q,), torch.int64, dev, here, stream)
    positions = _out(positions, "positions", (total_q,), i32, dev, here, stream)
    used = _out(used, "used", (1,), i32, dev, here, stream)
    args = _PLAN_ARGS.pack(B, total_q, page_size, width, n_prefix, fs[0], *lens, cu_q_lens.data_ptr(),
                           slot_mapping.data_ptr(), positions.data_ptr(), used.data_ptr())
    status = lib().dsa_page_plan(args, _stream_of(here, stream))
    if status != DSA_OK:
        raise DsaError(status, "dsa_page_plan")
    results = (cu_q_lens, slot_mapping, positions, used)
    if stream is not None:
        _hold(stream, (q_lens, seq_lens, block_tables, free_pages, prefix_pages) + results, results)
    return results


def dsa_mla_cache_append(c_kv: torch.Tensor, k_rope: torch.Tensor, slot_mapping: torch.Tensor, cache_c: torch.Tensor,
                         cache_r: torch.Tensor, *, norm_weight: Optional[torch.Tensor] = None,
                         norm_eps: float = 1e-6, rope_cos: Optional[torch.Tensor] = None,
                         rope_sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                         rope_interleaved: bool = False, stream=None) -> None:
    """This step's latent rows into the paged cache, in place: c_kv [n, 512] (root-mean-square
    norm times norm_weight [512] fp32, when given) into cache_c [num_pages, page_size, 512]
    and k_rope [n, 64] (turned by row positions[t] of rope_cos / rope_sin [rows, 32] fp32,
    when given; row t without positions) into cache_r [num_pages, page_size, 64], at the slots
    slot_mapping [n] (int64, page * page_size + row; negative = skip).  c_kv and k_rope may be
    views of one [n, 576] projection output."""
    if not (c_kv.dim() == k_rope.dim() == 2 and cache_c.dim() == 3 and (rope_cos is None or rope_cos.dim() == 2)):
        _expect([(c_kv, "c_kv", (None, None)), (k_rope, "k_rope", (None, None)),
                 (cache_c, "cache_c", (None, None, None)), (rope_cos, "rope_cos", (None, None))])
    n, R = c_kv.shape
    rd = k_rope.shape[1]
    num_pages, page_size = cache_c.shape[:2]
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("rope_cos and rope_sin go together")
    rows = 0 if rope_cos is None else rope_cos.shape[0]
    table = (rows, rd // 2)
    if not (k_rope.shape[0] == n and slot_mapping.shape == (n,) and cache_c.shape[2] == R
            and cache_r.shape == (num_pages, page_size, rd) and (norm_weight is None or norm_weight.shape == (R,))
            and (rope_cos is None or rope_cos.shape == rope_sin.shape == table)
            and (positions is None or positions.shape == (n,))):
        _expect([(k_rope, "k_rope", (n, rd)), (slot_mapping, "slot_mapping", (n,)),
                 (cache_c, "cache_c", (num_pages, page_size, R)), (cache_r, "cache_r", (num_pages, page_size, rd)),
                 (norm_weight, "norm_weight", (R,)), (rope_cos, "rope_cos", table), (rope_sin, "rope_sin", table),
                 (positions, "positions", (n,))])
    f32, bf16, here = torch.float32, torch.bfloat16, _here(cache_c)
    args = _APPEND_ARGS.pack(
        n, R, rd, page_size, num_pages, 1 if rope_interleaved else 0, rows, norm_eps, _rows(c_kv, "c_kv", here),
        _rows(k_rope, "k_rope", here), c_kv.stride(0), k_rope.stride(0),
        _ptr(slot_mapping, "slot_mapping", torch.int64, here), _ptr(norm_weight, "norm_weight", f32, here),
        _ptr(rope_cos, "rope_cos", f32, here), _ptr(rope_sin, "rope_sin", f32, here),
        _ptr(positions, "positions", torch.int32, here), _ptr(cache_c, "cache_c", bf16, here),
        _ptr(cache_r, "cache_r", bf16, here))
    status = lib().dsa_mla_cache_append(args, _stream_of(here, stream))
    if status != DSA_OK:
        raise DsaError(status, "dsa_mla_cache_append")
    if stream is not None:
        _hold(stream, (c_kv, k_rope, slot_mapping, cache_c, cache_r, norm_weight, rope_cos, rope_sin, positions))


def dsa_prefix_mla_workspace_size(B: int, total_q: int, H: int, *, prefix_len: int) -> int:
    """Bytes of workspace that dsa_prefix_mla takes for a batch of these sizes on the current device."""
    need = ctypes.c_size_t(0)
    args = _PREFIX_ARGS.pack(B, total_q, H, 512, 64, 64, 0, 0, prefix_len, -(-prefix_len // 64), 1.0, *[0] * 16)
    _check(lib().dsa_prefix_mla_workspace_size(args, ctypes.byref(need)), "dsa_prefix_mla_workspace_size")
    return int(need.value)


def dsa_prefix_mla(q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, prefix_pages=None, *,
                   prefix_len: int, scale: float, out=None, lse=None, workspace=None, stream=None):
    """Latent attention of a batch whose sequences share their first prefix_len tokens (their
    pages in prefix_pages; the rest through block_tables): (out [total_q, H, 512] bf16,
    lse [total_q, H] fp32, the natural logarithm of the sum of exponentials).  q_nope and
    q_rope may be views of one [total_q, H, 576] tensor.  out, lse and the workspace
    (dsa_prefix_mla_workspace_size bytes) are allocated when not given."""
    qs, rs, cs, bs = q_nope.shape, q_rope.shape, cache_c.shape, block_tables.shape
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    n_prefix = 0 if prefix_pages is None else prefix_pages.shape[0] if prefix_pages.dim() == 1 else -1
    if len(qs) != 3 or len(rs) != 3 or len(cs) != 3 or len(bs) != 2 or B < 0 or n_prefix < 0:
        _expect([(q_nope, "q_nope", (None, None, None)), (q_rope, "q_rope", (None, None, None)),
                 (cache_c, "cache_c", (None, None, None)), (seq_lens, "seq_lens", (None,)),
                 (block_tables, "block_tables", (None, None)), (prefix_pages, "prefix_pages", (None,))])
    T, H, R = qs
    rd = rs[2]
    num_pages, page_size, row = cs
    if (row != R or rs != (T, H, rd) or cache_r.shape != (num_pages, page_size, rd) or bs[0] != B
            or cu_q_lens.shape != (B + 1,)):
        _expect([(q_rope, "q_rope", (T, H, rd)), (cache_c, "cache_c", (num_pages, page_size, R)),
                 (cache_r, "cache_r", (num_pages, page_size, rd)), (block_tables, "block_tables", (B, None)),
                 (cu_q_lens, "cu_q_lens", (B + 1,))])
    i32, bf16, dev, here = torch.int32, torch.bfloat16, cache_c.device, _here(cache_c)
    sizes = (B, T, H, R, rd, page_size, num_pages, bs[1], prefix_len, n_prefix, scale)
    qt, qh, _ = q_nope.stride()
    rt, rh, _ = q_rope.stride()
    tensors = (_rows(q_nope, "q_nope", here), _rows(q_rope, "q_rope", here), qt, qh, rt, rh,
               _ptr(cache_c, "cache_c", bf16, here), _ptr(cache_r, "cache_r", bf16, here),
               _ptr(prefix_pages, "prefix_pages", i32, here), _ptr(block_tables, "block_tables", i32, here),
               _ptr(cu_q_lens, "cu_q_lens", i32, here), _ptr(seq_lens, "seq_lens", i32, here))
    out = _out(out, "out", (T, H, R), bf16, dev, here, stream)
    lse = _out(lse, "lse", (T, H), torch.float32, dev, here, stream)
    L = lib()
    if workspace is None:
        need = ctypes.c_size_t(0)
        status = L.dsa_prefix_mla_workspace_size(_PREFIX_ARGS.pack(*sizes, *tensors, 0, 0, 0, 0), ctypes.byref(need))
        if status != DSA_OK:
            raise DsaError(status, "dsa_prefix_mla_workspace_size")
        room = need.value or 16
        workspace = _new(room, torch.uint8, dev, stream)
    else:
        room = workspace.numel() * workspace.element_size()
    args = _PREFIX_ARGS.pack(*sizes, *tensors, out.data_ptr(), lse.data_ptr(), _dev(workspace, "workspace"), room)
    status = L.dsa_prefix_mla(args, _stream_of(here, stream))
    if status != DSA_OK:
        raise DsaError(status, "dsa_prefix_mla")
    if stream is not None:
        _hold(stream, (q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, prefix_pages, out, lse,
                       workspace), (out, lse))
    return out, lse


def dsa_test_arm_score_timeout(limit_ns: int) -> None:
    """Failure-path test hook: the next score-kernel launch of this host thread first
    waits up to limit_ns on a barrier nothing completes, then records DSA_ERR_TIMEOUT,
    drains and returns (its outputs are unspecified).  0 disarms."""
    _check(lib().dsa_test_arm_score_timeout(int(limit_ns)), "dsa_test_arm_score_timeout")


def dsa_test_arm_prefix_mla_timeout(site: int, at: int, limit_ns: int) -> None:
    """The same for the attention kernel of the next dsa_prefix_mla: a wait of one role runs out (1 MMAs
    before block `at`, 2 keys, 3 values, 4 queries before piece `at`, 5 softmax; + 8 in the odd CTAs)."""
    _check(lib().dsa_test_arm_prefix_mla_timeout(int(site), int(at), int(limit_ns)),
           "dsa_test_arm_prefix_mla_timeout")


def dsa_check_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status (DSA_OK, ...)."""
    return int(lib().dsa_check_device_status(_stream_ptr(stream)))


def dsa_clock_sample(n_ctas: int, stream=None):
    """Device tensor [n_ctas, 3] int64 of (SM id, SM cycle counter, global ns timer), one
    row per one-thread block; two samples bracket an interval (diagnostic)."""
    with _on(stream):
        out = torch.empty((n_ctas, 3), dtype=torch.int64, device="cuda")
    _check(lib().dsa_clock_sample(out.data_ptr(), int(n_ctas), _stream_ptr(stream)), "dsa_clock_sample")
    _hold(stream, (), (out,))
    return out


# ---- host helpers (GLM5 TensorCast adaptation design) -----------------------------

def resolve_topk_limit(explicit=None, indexer=None, config=None, indexer_config=None) -> int:
    """top-k width in the order of section "Sparse MLA 配置兼容": an explicit value, then
    the indexer's own topk_limit, then topk_limit on the attention / indexer config, then
    the GLM5-style index_topk; AttributeError("topk_limit") when none exists."""
    if explicit is not None:
        return int(explicit)
    if indexer is not None and getattr(indexer, "topk_limit", None) is not None:
        return int(indexer.topk_limit)
    for cfg in (config, indexer_config):
        if cfg is not None and getattr(cfg, "topk_limit", None) is not None:
            return int(cfg.topk_limit)
    for cfg in (config, indexer_config):
        if cfg is not None and getattr(cfg, "index_topk", None) is not None:
            return int(cfg.index_topk)
    raise AttributeError("topk_limit")


def extend_indexer_types_for_mtp(indexer_types: Sequence[str], num_mtp_layers: int) -> list:
    """Append one 'full' per MTP block (an MTP block cannot consume the main stack's
    top-k, section "GLM-5.2 IndexShare"); an empty list or zero MTP layers is unchanged."""
    types = list(indexer_types)
    if not types or num_mtp_layers <= 0:
        return types
    return types + ["full"] * int(num_mtp_layers)


# ---- no-allocation variant ----------------------------------------------------------

DSA_STATIC_WORKSPACE_BYTES = 24 << 20


def dsa_indexer_static(q, w, k_cache, cu_q_lens, seq_lens, block_tables, *, max_seq_len: int, topk_limit: int,
                       k_out: Optional[int] = None, q_scale=None, k_scale_cache=None, topk=None,
                       order: int = DSA_ORDER_SCORE, stream=None) -> torch.Tensor:
    """dsa_indexer without a workspace, for callers that cannot allocate device memory
    (plugin hosts that only pass tensors, serving loops that forbid allocation during a
    step).  The library keeps the scratch in a fixed device array of
    DSA_STATIC_WORKSPACE_BYTES; larger problems raise DsaError(DSA_ERR_WORKSPACE).
    Calls that overlap on the GPU share that array and must be serialised."""
    with _on(stream):
        a, keep = make_indexer_args(q, w, k_cache, cu_q_lens, seq_lens, block_tables, max_seq_len=max_seq_len,
                                    topk_limit=topk_limit, k_out=k_out, q_scale=q_scale,
                                    k_scale_cache=k_scale_cache, topk=topk,
                                    workspace=torch.empty(0, dtype=torch.uint8, device=q.device), order=order)
    a.workspace, a.workspace_bytes = None, 0
    fn = lib().dsa_indexer_static
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(dsa_indexer_args), ctypes.c_void_p]
    _check(fn(ctypes.byref(a), _stream_ptr(stream)), "dsa_indexer_static")
    _hold(stream, keep, (keep[8],))
    return keep[8]

"""ctypes binding of libfp2.so (include/fp2.h).  Argument marshalling only.

Every step of the attention path runs inside the CUDA library; PyTorch is used
here only to hand device pointers and the current stream to it.  Loading fails
loudly when the library has not been built.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# FP2_LIBRARY selects another build of the same library for this process (the tests use it to
# run with libfp2_checked.so); by default libfp2.so next to this file.
LIB_PATH = os.environ.get("FP2_LIBRARY") or os.path.join(_HERE, "libfp2.so")
CHECKED_LIB_PATH = os.path.join(_HERE, "libfp2_checked.so")

FP2_OK, FP2_ERR_INVALID_ARG, FP2_ERR_UNSUPPORTED, FP2_ERR_WORKSPACE_TOO_SMALL = 0, 1, 2, 3
FP2_ERR_CUDA, FP2_ERR_DEVICE_BOUNDS, FP2_ERR_TIMEOUT, FP2_ERR_CHECK_FAILED = 4, 5, 6, 7
FP2_F32, FP2_BF16, FP2_E4M3 = 0, 1, 2
FP2_DEV_PAGE_OOB, FP2_DEV_INDEX_OOB, FP2_DEV_CAPACITY, FP2_DEV_TIMEOUT, FP2_DEV_CHECK = 0x1, 0x2, 0x4, 0x8, 0x10
FP2_DEV_LEN_OOB, FP2_DEV_SLOT_OOB = 0x20, 0x40
FP2_BUILD_CHECKED = 0x1
FP2_MAX_SEQS, FP2_MAX_BLOCKS = 512, 4096
FP2_MAX_DRAFT, FP2_MAX_CACHE_LEN = 64, 524288

STATUS_NAMES = {0: "FP2_OK", 1: "FP2_ERR_INVALID_ARG", 2: "FP2_ERR_UNSUPPORTED", 3: "FP2_ERR_WORKSPACE_TOO_SMALL",
                4: "FP2_ERR_CUDA", 5: "FP2_ERR_DEVICE_BOUNDS", 6: "FP2_ERR_TIMEOUT", 7: "FP2_ERR_CHECK_FAILED"}

EXPORTED = ("fp2_workspace_query", "fp2_workspace_size", "fp2_pool", "fp2_discover", "fp2_attend", "fp2_prefill",
            "fp2_get_device_status", "fp2_last_error", "fp2_version", "fp2_discover_static", "fp2_debug_set",
            "fp2_build_flags", "fp2_rotate", "fp2_decode_workspace", "fp2_tree_attend", "fp2_key_mass",
            "fp2_evict_workspace", "fp2_evict")
FP2_DEBUG_WAIT_LIMIT_NS, FP2_DEBUG_WITHHOLD_K_TILE, FP2_DEBUG_MISCOUNT_LOAD, FP2_DEBUG_LATE_V_TILE = 1, 2, 3, 4
FP2_STATIC_SCRATCH_BYTES = 8 << 20
FP2_STREAM_NONE = ctypes.c_void_p(-1).value


class fp2_problem(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("cu_seqlens_q_host", ctypes.POINTER(ctypes.c_int32)),
        ("cu_seqlens_k_host", ctypes.POINTER(ctypes.c_int32)),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int),
        ("q_descale", ctypes.c_float), ("k_descale", ctypes.c_float), ("v_descale", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride_tok", ctypes.c_int64), ("kv_stride_tok", ctypes.c_int64),
        ("page_table", ctypes.c_void_p),
        ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("kv_prefix_pooled", ctypes.c_int32),
    ]


class fp2_sparse_params(ctypes.Structure):
    _fields_ = [
        ("block_size", ctypes.c_int32), ("alpha", ctypes.c_float), ("sink_blocks", ctypes.c_int32),
        ("window_blocks", ctypes.c_int32), ("last_n_blocks", ctypes.c_int32), ("min_sparse_len", ctypes.c_int32),
        ("mean_correction", ctypes.c_int32), ("kv_splits", ctypes.c_int32),
    ]


class fp2_pooled(ctypes.Structure):
    _fields_ = [("qbar", ctypes.c_void_p), ("kbar", ctypes.c_void_p), ("vbar", ctypes.c_void_p),
                ("kbar_mma", ctypes.c_void_p), ("vbar_mma", ctypes.c_void_p), ("v16", ctypes.c_void_p)]


class fp2_index(ctypes.Structure):
    _fields_ = [("row_ptr", ctypes.c_void_p), ("col_idx", ctypes.c_void_p), ("col_capacity", ctypes.c_int64)]


class fp2_workspace(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64), ("total_kv_tokens", ctypes.c_int64), ("total_q_blocks", ctypes.c_int64),
        ("total_kv_blocks", ctypes.c_int64), ("index_rows", ctypes.c_int64), ("col_capacity", ctypes.c_int64),
        ("qbar_bytes", ctypes.c_size_t), ("kbar_bytes", ctypes.c_size_t), ("vbar_bytes", ctypes.c_size_t),
        ("kbar_mma_bytes", ctypes.c_size_t), ("vbar_mma_bytes", ctypes.c_size_t),
        ("row_ptr_bytes", ctypes.c_size_t), ("col_idx_bytes", ctypes.c_size_t),
        ("discover_scratch_bytes", ctypes.c_size_t), ("scratch_bytes", ctypes.c_size_t),
        ("prefill_scratch_bytes", ctypes.c_size_t), ("v16_bytes", ctypes.c_size_t),
    ]


class fp2_cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("dtype", ctypes.c_int), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("stride_tok", ctypes.c_int64), ("stride_outer", ctypes.c_int64),
        ("num_outer", ctypes.c_int32), ("rows", ctypes.c_int32),
        ("page_table", ctypes.c_void_p), ("max_pages_per_seq", ctypes.c_int32),
    ]


class fp2_rotation(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride_tok", ctypes.c_int64), ("k_stride_tok", ctypes.c_int64), ("v_stride_tok", ctypes.c_int64),
        ("positions", ctypes.c_void_p),
        ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("inv_freq_host", ctypes.POINTER(ctypes.c_double)), ("rope_scale", ctypes.c_float),
        ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
        ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p),
        ("q_out_stride_tok", ctypes.c_int64), ("kv_out_stride_tok", ctypes.c_int64),
        ("slots", ctypes.c_void_p), ("num_slots", ctypes.c_int64),
        ("q_descale", ctypes.c_float), ("k_descale", ctypes.c_float), ("v_descale", ctypes.c_float),
    ]


class fp2_decode(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("cu_seqlens_q_host", ctypes.POINTER(ctypes.c_int32)),
        ("num_q_heads", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("q_stride_tok", ctypes.c_int64),
        ("q_descale", ctypes.c_float), ("k_descale", ctypes.c_float), ("v_descale", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("cache", fp2_cache),
        ("kv_len", ctypes.c_void_p), ("max_kv_len", ctypes.c_int32),
        ("tree_mask", ctypes.c_void_p),
    ]


class fp2_eviction(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("src", fp2_cache), ("dst", fp2_cache),
        ("kv_len", ctypes.c_void_p), ("max_kv_len", ctypes.c_int32),
        ("mass", ctypes.c_void_p), ("mass_stride", ctypes.c_int64),
        ("budget", ctypes.c_int32), ("sink", ctypes.c_int32), ("window", ctypes.c_int32),
        ("mass_out", ctypes.c_void_p), ("kept", ctypes.c_void_p), ("kv_len_out", ctypes.c_void_p),
    ]


class FP2Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfp2.so (once).  Raises when it is missing: there is no fallback path."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with block_sparse_long_pooled_b200.build.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.fp2_workspace_query.argtypes = [P(fp2_problem), P(fp2_sparse_params), P(fp2_workspace)]
    lib.fp2_workspace_size.argtypes = [P(fp2_problem), P(fp2_sparse_params), P(sz), P(sz), P(sz)]
    lib.fp2_pool.argtypes = [P(fp2_problem), P(fp2_sparse_params), P(fp2_pooled), vp, sz, vp]
    lib.fp2_discover.argtypes = [P(fp2_problem), P(fp2_sparse_params), P(fp2_pooled), P(fp2_index), vp, sz, vp]
    lib.fp2_attend.argtypes = [P(fp2_problem), P(fp2_sparse_params), P(fp2_pooled), P(fp2_index), vp, vp, vp, sz, vp]
    lib.fp2_prefill.argtypes = [P(fp2_problem), P(fp2_sparse_params), vp, vp, vp, sz, vp]
    lib.fp2_get_device_status.argtypes = [vp, P(ctypes.c_uint32)]
    lib.fp2_discover_static.argtypes = [P(fp2_problem), P(fp2_sparse_params), P(fp2_pooled), P(fp2_index), vp, vp]
    lib.fp2_rotate.argtypes = [P(fp2_rotation), vp, vp]
    lib.fp2_decode_workspace.argtypes = [P(fp2_decode), P(sz)]
    lib.fp2_tree_attend.argtypes = [P(fp2_decode), vp, vp, vp, sz, vp]
    lib.fp2_key_mass.argtypes = [P(fp2_decode), vp, vp, vp, ctypes.c_int64, vp, ctypes.c_float, vp, sz, vp]
    lib.fp2_evict_workspace.argtypes = [P(fp2_eviction), P(sz)]
    lib.fp2_evict.argtypes = [P(fp2_eviction), vp, sz, vp]
    for name in ("fp2_workspace_query", "fp2_workspace_size", "fp2_pool", "fp2_discover", "fp2_attend", "fp2_prefill",
                 "fp2_get_device_status", "fp2_discover_static", "fp2_rotate", "fp2_decode_workspace",
                 "fp2_tree_attend", "fp2_key_mass", "fp2_evict_workspace", "fp2_evict"):
        getattr(lib, name).restype = ctypes.c_int
    lib.fp2_debug_set.argtypes = [ctypes.c_int32, ctypes.c_int64]
    lib.fp2_debug_set.restype = ctypes.c_int
    lib.fp2_last_error.argtypes = []
    lib.fp2_last_error.restype = ctypes.c_char_p
    lib.fp2_version.argtypes = []
    lib.fp2_version.restype = ctypes.c_int32
    lib.fp2_build_flags.argtypes = []
    lib.fp2_build_flags.restype = ctypes.c_uint32
    _lib = lib
    return lib


def _check(status: int):
    if status != FP2_OK:
        raise FP2Error(status, load_library().fp2_last_error().decode())


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(stream) if isinstance(stream, int) else int(stream.cuda_stream)


# ------------------------------------------------------------------ problem description

@dataclasses.dataclass
class Problem:
    """An fp2_problem plus the host arrays and tensors it points into (kept alive here)."""
    struct: fp2_problem
    cu_seqlens: np.ndarray
    keep: tuple
    cu_seqlens_k: Optional[np.ndarray] = None


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: FP2_F32, torch.bfloat16: FP2_BF16, torch.float8_e4m3fn: FP2_E4M3,
            torch.uint8: FP2_E4M3}[t.dtype]


def make_problem(q, k, v, cu_seqlens, num_kv_heads: int, q_descale: float = 1.0, k_descale: float = 1.0,
                 v_descale: float = 1.0, softmax_scale: float = 0.0, page_table=None,
                 num_pages: int = 0, cu_seqlens_k=None, kv_prefix_pooled: bool = False) -> Problem:
    """q: [T, Hq, d]; k, v: [Tk, Hkv, d] or a paged cache [P, page_size, Hkv, d] with page_table
    [num_seqs, max_pages] (int32, device).  cu_seqlens: host int sequence [num_seqs + 1] of query
    offsets; cu_seqlens_k: key offsets when the queries are chunks at the end of their sequences
    (chunked prefill), else None.  kv_prefix_pooled: the pooled prefix K/V blocks are already in
    the pooled buffers (see include/fp2.h)."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    cuk = None if cu_seqlens_k is None else np.ascontiguousarray(np.asarray(cu_seqlens_k, dtype=np.int32))
    s = fp2_problem()
    s.num_seqs = len(cu) - 1
    s.cu_seqlens_q_host = cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    s.cu_seqlens_k_host = s.cu_seqlens_q_host if cuk is None else cuk.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    s.kv_prefix_pooled = 1 if kv_prefix_pooled else 0
    s.num_q_heads = q.shape[1]
    s.num_kv_heads = num_kv_heads
    s.head_dim = q.shape[2]
    s.dtype = _dtype_code(q)
    s.q_descale, s.k_descale, s.v_descale = q_descale, k_descale, v_descale
    s.softmax_scale = softmax_scale
    s.q, s.k, s.v = _ptr(q), _ptr(k), _ptr(v)
    s.q_stride_tok = q.stride(0)
    if page_table is not None:
        s.kv_stride_tok = k.stride(1)
        s.page_table = _ptr(page_table)
        s.page_size = k.shape[1]
        s.max_pages_per_seq = page_table.shape[1]
        s.num_pages = num_pages or k.shape[0]
    else:
        s.kv_stride_tok = k.stride(0)
        s.page_table = None
    return Problem(struct=s, cu_seqlens=cu, keep=(q, k, v, page_table), cu_seqlens_k=cuk)


def make_params(block_size: int, alpha: float = 0.1, sink_blocks: int = 2, window_blocks: int = 4,
                last_n_blocks: int = 0, min_sparse_len: int = 0, mean_correction: bool = True,
                kv_splits: int = 0) -> fp2_sparse_params:
    return fp2_sparse_params(block_size, alpha, sink_blocks, window_blocks, last_n_blocks, min_sparse_len,
                             1 if mean_correction else 0, kv_splits)


# ------------------------------------------------------------------ the C entry points

def fp2_workspace_query(problem: Problem, params: fp2_sparse_params) -> fp2_workspace:
    ws = fp2_workspace()
    _check(load_library().fp2_workspace_query(ctypes.byref(problem.struct), ctypes.byref(params), ctypes.byref(ws)))
    return ws


def fp2_workspace_size(problem: Problem, params: fp2_sparse_params) -> tuple:
    """(pooled_bytes, index_bytes, scratch_bytes): the totals for carving the pooled buffers and the
    index from one allocation each (256-byte aligned offsets), and the scratch size."""
    pooled, index, scratch = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load_library().fp2_workspace_size(ctypes.byref(problem.struct), ctypes.byref(params), ctypes.byref(pooled),
                                             ctypes.byref(index), ctypes.byref(scratch)))
    return pooled.value, index.value, scratch.value


def fp2_pool(problem: Problem, params, pooled: fp2_pooled, scratch, stream=None):
    _check(load_library().fp2_pool(ctypes.byref(problem.struct), ctypes.byref(params), ctypes.byref(pooled),
                                   _ptr(scratch), scratch.numel() * scratch.element_size(), _stream_handle(stream)))


def fp2_discover(problem: Problem, params, pooled: fp2_pooled, index: fp2_index, scratch, stream=None):
    _check(load_library().fp2_discover(ctypes.byref(problem.struct), ctypes.byref(params), ctypes.byref(pooled),
                                       ctypes.byref(index), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                       _stream_handle(stream)))


def fp2_attend(problem: Problem, params, pooled: fp2_pooled, index: fp2_index, out, lse, scratch, stream=None):
    _check(load_library().fp2_attend(ctypes.byref(problem.struct), ctypes.byref(params), ctypes.byref(pooled),
                                     ctypes.byref(index), _ptr(out), _ptr(lse), _ptr(scratch),
                                     scratch.numel() * scratch.element_size(), _stream_handle(stream)))


def fp2_prefill(problem: Problem, params, out, lse, scratch, stream=None):
    _check(load_library().fp2_prefill(ctypes.byref(problem.struct), ctypes.byref(params), _ptr(out), _ptr(lse),
                                      _ptr(scratch), scratch.numel() * scratch.element_size(),
                                      _stream_handle(stream)))


def fp2_discover_static(problem: Problem, params, pooled: fp2_pooled, index: fp2_index, status_dev=None,
                        stream=None):
    """fp2_discover without a scratch argument, for callers that cannot allocate device memory where
    they run discovery.  The library keeps the scratch in its own static device buffer (shared by all
    calls on a GPU: do not overlap calls).  status_dev: optional int32/uint32 device tensor of >= 1
    element that receives the call's FP2_DEV_* status word."""
    _check(load_library().fp2_discover_static(ctypes.byref(problem.struct), ctypes.byref(params),
                                              ctypes.byref(pooled), ctypes.byref(index), _ptr(status_dev),
                                              _stream_handle(stream)))


def fp2_get_device_status(scratch) -> tuple:
    """(status code, raw FP2_DEV_* bits); call after synchronising the stream."""
    bits = ctypes.c_uint32(0)
    st = load_library().fp2_get_device_status(_ptr(scratch), ctypes.byref(bits))
    return st, int(bits.value)


def fp2_debug_set(key: int, value: int):
    """Testing hook (process-wide): FP2_DEBUG_WAIT_LIMIT_NS, FP2_DEBUG_WITHHOLD_K_TILE, and in
    checked builds FP2_DEBUG_MISCOUNT_LOAD or FP2_DEBUG_LATE_V_TILE."""
    _check(load_library().fp2_debug_set(int(key), int(value)))


def fp2_last_error() -> str:
    return load_library().fp2_last_error().decode()


def fp2_version() -> int:
    return int(load_library().fp2_version())


def fp2_build_flags() -> int:
    """FP2_BUILD_* bits of the loaded library (FP2_BUILD_CHECKED for libfp2_checked.so)."""
    return int(load_library().fp2_build_flags())


# ------------------------------------------------------------------ buffer helpers (torch allocations)

def alloc_pooled(ws: fp2_workspace, problem: Problem, device):
    """Device buffers for fp2_pooled, as torch tensors; returns (struct, dict of tensors)."""
    import torch
    s = problem.struct
    nq, nk, Hq, Hkv, D = ws.total_q_blocks, ws.total_kv_blocks, s.num_q_heads, s.num_kv_heads, s.head_dim
    mma_dtype = {FP2_F32: torch.float32, FP2_BF16: torch.bfloat16, FP2_E4M3: torch.uint8}[s.dtype]
    # the V side of the PV product is f16 for E4M3 inputs (pooled vbar and the copy of V)
    v_dtype = torch.float16 if s.dtype == FP2_E4M3 else mma_dtype
    t = {
        "qbar": torch.empty((nq, Hq, D), dtype=torch.float32, device=device),
        "kbar": torch.empty((nk, Hkv, D), dtype=torch.float32, device=device),
        "vbar": torch.empty((nk, Hkv, D), dtype=torch.float32, device=device),
        "kbar_mma": torch.empty((nk, Hkv, D), dtype=mma_dtype, device=device),
        "vbar_mma": torch.empty((nk, Hkv, D), dtype=v_dtype, device=device),
    }
    if s.dtype == FP2_E4M3:
        t["v16"] = torch.empty((ws.total_kv_tokens, Hkv, D), dtype=torch.float16, device=device)
    return pooled_struct(t), t


def pooled_struct(t: dict) -> fp2_pooled:
    """fp2_pooled from a dict of tensors (qbar, kbar, vbar, kbar_mma, vbar_mma and, for E4M3, v16), which it keeps
    alive."""
    s = fp2_pooled(*(_ptr(t.get(k)) for k in ("qbar", "kbar", "vbar", "kbar_mma", "vbar_mma", "v16")))
    s.keep = tuple(t.values())
    return s


def index_struct(row_ptr, col_idx) -> fp2_index:
    """fp2_index of two tensors, which it keeps alive."""
    s = fp2_index(_ptr(row_ptr), _ptr(col_idx), int(col_idx.numel()))
    s.keep = (row_ptr, col_idx)
    return s


def alloc_index(ws: fp2_workspace, device):
    import torch
    row_ptr = torch.empty(ws.index_rows + 1, dtype=torch.int32, device=device)
    col_idx = torch.empty(max(1, ws.col_capacity), dtype=torch.int32, device=device)
    return index_struct(row_ptr, col_idx), {"row_ptr": row_ptr, "col_idx": col_idx}


def alloc_scratch(nbytes: int, device):
    import torch
    return torch.empty(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


def out_dtype(problem: Problem):
    import torch
    return torch.float32 if problem.struct.dtype == FP2_F32 else torch.bfloat16


# ------------------------------------------------------------------ serving: positions, decode, eviction

@dataclasses.dataclass
class Rope:
    """Frequencies of a rotary embedding: pair i turns by position * inv_freq[i] radians."""
    inv_freq: np.ndarray            # float64 [rotary_dim / 2]
    interleaved: bool = False       # pairs (2i, 2i+1); else (i, i + rotary_dim/2)
    scale: float = 1.0              # factor on cosine and sine


def make_rope(inv_freq, interleaved: bool = False, scale: float = 1.0) -> Rope:
    """inv_freq: host sequence or array; its length is half the rotary dimension (a multiple of 8)."""
    f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
    if f.ndim != 1:
        raise ValueError("inv_freq must be one-dimensional")
    return Rope(f, bool(interleaved), float(scale))


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_len: int = 8192, low: float = 1.0, high: float = 4.0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0) -> tuple:
    """(inverse frequencies, factor on cosine and sine) for make_rope.

    scaling None: base^(-2i/rotary_dim).  "linear": divided by factor.  "ntk": the base is raised so
    that the slowest pair is slowed down by factor.  "llama3": pairs that turn less than `low` times in
    original_len are divided by factor, those above `high` times kept, linear in the turns between.
    "yarn": kept above beta_fast turns, divided below beta_slow, linear in the pair's index between,
    and cosine and sine scaled by 0.1 ln(factor) + 1."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be a positive even number")
    if not factor > 0 or not base > 1:
        raise ValueError("factor must be positive and base above 1")
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / max(rotary_dim - 2, 1))
    f = base ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    if scaling in (None, "none", "ntk"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "llama3":
        t = np.clip((original_len * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        return f * ((1 - t) / factor + t), 1.0
    if scaling == "yarn":
        def pair(turns):   # index of the pair that turns that often in original_len
            return rotary_dim * np.log(original_len / (turns * 2 * np.pi)) / (2 * np.log(base))
        first, last = max(np.floor(pair(beta_fast)), 0), min(np.ceil(pair(beta_slow)), rotary_dim - 1)
        t = np.clip((np.arange(rotary_dim // 2) - first) / max(last - first, 0.001), 0.0, 1.0)
        return f * (1 - t + t / factor), float(0.1 * np.log(factor) + 1.0) if factor > 1 else 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


class _Handle:
    """A C struct, the tensors it points into (kept alive here) and the device they are on.  The calls on
    it last microseconds, so what they need of torch and of the library is looked up once."""

    def __init__(self, struct, tensors, arrays=()):
        import torch
        self.struct, self.ref = struct, ctypes.byref(struct)
        self.keep = (tuple(tensors), tuple(arrays))
        devices = {t.device for t in tensors if t is not None}
        if len(devices) > 1:
            raise ValueError(f"tensors on different devices: {sorted(map(str, devices))}")
        self.device = devices.pop()
        self.cuda = self.device.type == "cuda"
        self.index = self.device.index if self.cuda else -1
        self.lib = load_library()
        if self.cuda:
            # current_stream(device).cuda_stream and current_device() without the objects around them
            self.raw_stream, self.current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            self.guard, self.alone = torch.cuda.device, torch.cuda.device_count() == 1

    def call(self, fn, args, stream):
        """The C entry point fn on this handle, on its device and (stream None) that device's current stream.
        Tensors of the host are refused."""
        if not self.cuda:       # host memory: the library's checks, and then its refusal
            status = fn(self.ref, *args, FP2_STREAM_NONE)
        else:
            raw = self.raw_stream(self.index) if stream is None else _stream_handle(stream)
            if self.alone or self.current() == self.index:
                status = fn(self.ref, *args, raw)
            else:
                with self.guard(self.index):
                    status = fn(self.ref, *args, raw)
        if status:
            _check(status)

    def pointer(self, t, dtype, shape, what: str):
        """data_ptr of a contiguous tensor of this handle's device, or None."""
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self.index:
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {self.device}")
        return t.data_ptr()

    def space(self, scratch):
        if scratch.get_device() != self.index:
            raise ValueError(f"scratch must be on {self.device}")
        return scratch.data_ptr(), scratch.nbytes


class Rotation(_Handle):
    pass


class Decode(_Handle):
    def __init__(self, struct, tensors, arrays=()):
        import torch
        super().__init__(struct, tensors, arrays)
        tokens, heads, dim = tensors[0].shape
        self.out_shape, self.lse_shape = (tokens, heads, dim), (heads, tokens)
        self.seqs, self.kv_heads, self.has_v = struct.num_seqs, struct.cache.num_kv_heads, bool(struct.cache.v)
        self.types = torch.float32 if struct.cache.dtype == FP2_F32 else torch.bfloat16, torch.float32, torch.int32


class Eviction(_Handle):
    pass


@dataclasses.dataclass
class Cache:
    """An fp2_cache and the tensors it points into."""
    struct: fp2_cache
    keep: tuple


def _head_rows(t, what: str, dims: int = 3):
    """Check that the last two dimensions of t, [..., heads, d], are dense."""
    if t.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions")
    if t.stride(-1) != 1 or (t.shape[-2] > 1 and t.stride(-2) != t.shape[-1]):
        raise ValueError(f"heads of {what} must be dense (strides (d, 1))")


def _expect(t, dtype, shape, what: str):
    if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _int32(x, what: str) -> int:
    """x, which a C int holds (ctypes would cut off what does not fit)."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{what} out of range")
    return x


def _stored_like(a, b) -> bool:
    return _dtype_code(a) == _dtype_code(b)


def make_cache(k, v=None, page_table=None) -> Cache:
    """k, v: [num_pages, page_size, Hkv, d] with page_table [num_seqs, max_pages] (int32), or without one
    [num_seqs, rows, Hkv, d].  v may be None for fp2_key_mass."""
    import torch
    _head_rows(k, "k", 4)
    if v is not None:
        _head_rows(v, "v", 4)
        if tuple(v.shape) != tuple(k.shape) or not _stored_like(k, v) or v.device != k.device:
            raise ValueError("k and v must agree in shape, dtype and device")
        if any(v.shape[i] > 1 and v.stride(i) != k.stride(i) for i in (0, 1)):
            raise ValueError("k and v must have the same strides")
    c = fp2_cache()
    c.k, c.v, c.dtype = _ptr(k), _ptr(v), _dtype_code(k)
    c.num_outer, c.rows, c.num_kv_heads, c.head_dim = k.shape
    hd = k.shape[2] * k.shape[3]
    c.stride_tok = k.stride(1) if k.shape[1] > 1 else hd
    c.stride_outer = k.stride(0) if k.shape[0] > 1 else c.rows * c.stride_tok
    if page_table is not None:
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous int32 tensor [num_seqs, max_pages]")
        if page_table.device != k.device:
            raise ValueError("page_table must be on the cache's device")
        c.page_table, c.max_pages_per_seq = _ptr(page_table), page_table.shape[1]
    return Cache(c, (k, v, page_table))


def _check_table(cache: Cache, num_seqs: int):
    table = cache.keep[2]
    if table is not None and table.shape[0] < num_seqs:
        raise ValueError("page_table has fewer rows than there are sequences")


def make_rotate(q, k, v, positions, rope: Optional[Rope], q_out, k_out, v_out, slots=None, q_norm=None, k_norm=None,
                norm_eps: float = 1e-6, q_descale: float = 1.0, k_descale: float = 1.0,
                v_descale: float = 1.0) -> Rotation:
    """q [T, Hq, d], k and v [T, Hkv, d] (views of one projection's output will do; q, or k and v, or v
    alone may be None); positions [T] int32; rope from make_rope, or None (norms and copies only).
    q_out [T, Hq, d]; k_out, v_out [rows, Hkv, d] or a paged cache [pages, page_size, Hkv, d], whose
    row slots[t] (int64, < 0: none) token t's K and V go to; without slots, row t."""
    import torch
    given = [(x, n) for x, n in ((q, "q"), (k, "k"), (v, "v")) if x is not None]
    if not given or (k is None and v is not None):
        raise ValueError("q or k must be given, and v only with k")
    first = given[0][0]
    T, d = first.shape[0], first.shape[-1]
    for x, n in given:
        _head_rows(x, n)
        if x.shape[0] != T or x.shape[2] != d or x.dtype != first.dtype:
            raise ValueError("q, k and v must agree in tokens, head_dim and dtype")
    if v is not None and v.shape[1] != k.shape[1]:
        raise ValueError("k and v must have the same heads")
    s = fp2_rotation()
    s.tokens, s.head_dim, s.in_dtype = T, d, _dtype_code(first)
    outs = [(q, q_out, "q_out"), (k, k_out, "k_out"), (v, v_out, "v_out")]
    outs = [(x, o, n) for x, o, n in outs if x is not None]
    if any(o is None for _, o, _ in outs):
        raise ValueError("every input needs its output")
    s.out_dtype = _dtype_code(outs[0][1])
    if any(_dtype_code(o) != s.out_dtype for _, o, _ in outs):
        raise ValueError("outputs must have one dtype")

    def stride(x):
        return x.stride(0) if x.shape[0] > 1 else x.shape[1] * x.shape[2]

    if q is not None:
        _head_rows(q_out, "q_out")
        if tuple(q_out.shape) != tuple(q.shape):
            raise ValueError("q_out must have q's shape")
        s.num_q_heads, s.q, s.q_stride_tok = q.shape[1], _ptr(q), stride(q)
        s.q_out, s.q_out_stride_tok = _ptr(q_out), stride(q_out)
    if k is not None:
        rows, steps = [], []
        for x, o, n in outs:
            if n == "q_out":        # (by name: q may be the tensor that k is)
                continue
            _head_rows(o, n, o.dim())
            if o.dim() not in (3, 4) or tuple(o.shape[-2:]) != tuple(x.shape[1:]):
                raise ValueError(f"{n} must be [rows, Hkv, d] or [pages, page_size, Hkv, d]")
            step = o.stride(-3) if o.shape[-3] > 1 else (o.stride(0) if o.dim() == 4 else o.shape[-2] * o.shape[-1])
            if o.dim() == 4 and o.shape[0] > 1 and o.stride(0) != o.shape[1] * step:
                raise ValueError(f"pages of {n} must follow each other without a gap")
            rows.append(o.shape[0] if o.dim() == 3 else o.shape[0] * o.shape[1])
            if rows[-1] > 1 and step < o.shape[-2] * o.shape[-1]:
                raise ValueError(f"rows of {n} overlap")
            steps.append(step)
        s.num_slots = min(rows)
        if len(set(steps)) != 1:
            raise ValueError("k_out and v_out must have the same token stride")
        s.num_kv_heads, s.k, s.k_stride_tok, s.k_out = k.shape[1], _ptr(k), stride(k), _ptr(k_out)
        s.kv_out_stride_tok = max(steps[0], k.shape[1] * d)
        if v is not None:
            s.v, s.v_stride_tok, s.v_out = _ptr(v), stride(v), _ptr(v_out)
    arrays = ()
    if rope is not None:
        arrays = (rope.inv_freq,)
        s.rotary_dim, s.interleaved, s.rope_scale = 2 * len(rope.inv_freq), int(rope.interleaved), rope.scale
        s.inv_freq_host = rope.inv_freq.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
        _expect(positions, torch.int32, (T,), "positions")
        s.positions = _ptr(positions)
    _expect(slots, torch.int64, (T,), "slots")
    _expect(q_norm, first.dtype, (d,), "q_norm")
    _expect(k_norm, first.dtype, (d,), "k_norm")
    s.slots, s.q_norm, s.k_norm, s.norm_eps = _ptr(slots), _ptr(q_norm), _ptr(k_norm), norm_eps
    s.q_descale, s.k_descale, s.v_descale = q_descale, k_descale, v_descale
    return Rotation(s, (q, k, v, positions if rope is not None else None, slots, q_norm, k_norm, q_out, k_out, v_out),
                    arrays)


def fp2_rotate(rotation: Rotation, status_dev=None, stream=None):
    """Head norms, rotary positions and cache append (include/fp2.h).  status_dev: optional int32/uint32
    device word that FP2_DEV_* bits are OR-ed into."""
    if status_dev is not None and (status_dev.element_size() != 4 or status_dev.numel() < 1 or
                                   status_dev.get_device() != rotation.index):
        raise ValueError(f"status_dev must be a 4-byte word on {rotation.device}")
    rotation.call(rotation.lib.fp2_rotate, (None if status_dev is None else status_dev.data_ptr(),), stream)


def make_decode(q, cache: Cache, cu_seqlens, kv_len, max_kv_len: int, num_kv_heads: Optional[int] = None,
                tree_mask=None, q_descale: float = 1.0, k_descale: float = 1.0, v_descale: float = 1.0,
                softmax_scale: float = 0.0) -> Decode:
    """q [T, Hq, d]: the new tokens of each sequence, cu_seqlens (host, [num_seqs + 1]) their offsets.
    kv_len [num_seqs] int32 on the device: keys per sequence, the new ones (already in the cache)
    included; max_kv_len: a bound on them.  tree_mask [T] int64 (bit b: the token sees new key b), or
    None: a chain."""
    import torch
    _head_rows(q, "q")
    c = cache.struct
    if num_kv_heads is not None and num_kv_heads != c.num_kv_heads:
        raise ValueError("num_kv_heads differs from the cache's")
    if q.shape[2] != c.head_dim or _dtype_code(q) != c.dtype:
        raise ValueError("q must have the cache's head_dim and dtype")
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    if cu.ndim != 1 or len(cu) < 2 or cu[-1] != q.shape[0]:
        raise ValueError("cu_seqlens must end at the number of tokens of q")
    _check_table(cache, len(cu) - 1)
    _expect(kv_len, torch.int32, (len(cu) - 1,), "kv_len")
    _expect(tree_mask, torch.int64, (q.shape[0],), "tree_mask")
    s = fp2_decode()
    s.num_seqs, s.cu_seqlens_q_host = len(cu) - 1, cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    s.num_q_heads, s.q = q.shape[1], _ptr(q)
    s.q_stride_tok = q.stride(0) if q.shape[0] > 1 else q.shape[1] * q.shape[2]
    s.q_descale, s.k_descale, s.v_descale, s.softmax_scale = q_descale, k_descale, v_descale, softmax_scale
    s.cache = c
    s.kv_len, s.max_kv_len, s.tree_mask = _ptr(kv_len), _int32(max_kv_len, "max_kv_len"), _ptr(tree_mask)
    return Decode(s, (q, kv_len, tree_mask, *cache.keep), (cu,))


def fp2_decode_workspace(decode: Decode) -> int:
    """Scratch bytes of fp2_tree_attend and fp2_key_mass (each its own where both calls' status is read)."""
    n = ctypes.c_size_t(0)
    _check(load_library().fp2_decode_workspace(decode.ref, ctypes.byref(n)))
    return n.value


def fp2_tree_attend(decode: Decode, out, lse, scratch, stream=None):
    """Attention of the new tokens over their caches.  out [T, Hq, d] bf16 (f32 over an F32 cache); lse
    [Hq, T] f32 or None."""
    if not decode.has_v:
        raise ValueError("the cache has no v")
    wide, f32, _ = decode.types
    decode.call(decode.lib.fp2_tree_attend, (decode.pointer(out, wide, decode.out_shape, "out"),
                                             decode.pointer(lse, f32, decode.lse_shape, "lse"),
                                             *decode.space(scratch)), stream)


def fp2_key_mass(decode: Decode, lse, mass_in, mass_out, scratch, decay: float = 1.0, mass_len=None, stream=None):
    """mass_out = decay * mass_in + the attention weight that each key receives from the new tokens.
    lse [Hq, T] from fp2_tree_attend; mass_in (or None: zero), mass_out [num_seqs, Hkv, >= max_kv_len]
    f32 (they may be one tensor); mass_len [num_seqs] int32: keys that mass_in covers, or None: all."""
    _, f32, i32 = decode.types
    shape = (decode.seqs, decode.kv_heads, mass_out.shape[-1])
    decode.call(decode.lib.fp2_key_mass, (decode.pointer(lse, f32, decode.lse_shape, "lse"),
                                          decode.pointer(mass_in, f32, shape, "mass_in"),
                                          decode.pointer(mass_out, f32, shape, "mass_out"), shape[2],
                                          decode.pointer(mass_len, i32, (decode.seqs,), "mass_len"), decay,
                                          *decode.space(scratch)), stream)


def make_evict(cache: Cache, kv_len, max_kv_len: int, mass, budget: int, sink: int, window: int, cache_out: Cache,
               mass_out, kept, kv_len_out) -> Eviction:
    """cache, kv_len [num_seqs] int32, mass [num_seqs, Hkv, >= max_kv_len] f32: the keys and their weights.
    cache_out gets the kept rows; mass_out [num_seqs, Hkv, budget] f32 and kept (int32, the same shape)
    their weights and old indexes, kv_len_out [num_seqs] int32 the new lengths."""
    import torch
    n, c = kv_len.shape[0], cache.struct
    _check_table(cache, n)
    _check_table(cache_out, n)
    _expect(kv_len, torch.int32, (n,), "kv_len")
    _expect(mass, torch.float32, (n, c.num_kv_heads, mass.shape[-1]), "mass")
    _expect(mass_out, torch.float32, (n, c.num_kv_heads, budget), "mass_out")
    _expect(kept, torch.int32, (n, c.num_kv_heads, budget), "kept")
    _expect(kv_len_out, torch.int32, (n,), "kv_len_out")
    s = fp2_eviction()
    s.num_seqs, s.src, s.dst = n, c, cache_out.struct
    s.kv_len, s.max_kv_len, s.mass, s.mass_stride = _ptr(kv_len), _int32(max_kv_len, "max_kv_len"), _ptr(mass), mass.shape[-1]
    s.budget, s.sink, s.window = _int32(budget, "budget"), _int32(sink, "sink"), _int32(window, "window")
    s.mass_out, s.kept, s.kv_len_out = _ptr(mass_out), _ptr(kept), _ptr(kv_len_out)
    return Eviction(s, (kv_len, mass, mass_out, kept, kv_len_out, *cache.keep, *cache_out.keep))


def fp2_evict_workspace(eviction: Eviction) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().fp2_evict_workspace(eviction.ref, ctypes.byref(n)))
    return n.value


def fp2_evict(eviction: Eviction, scratch, stream=None):
    """Keep each (sequence, KV head)'s heaviest keys, in another cache (include/fp2.h)."""
    eviction.call(eviction.lib.fp2_evict, eviction.space(scratch), stream)

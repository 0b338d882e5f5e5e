"""ctypes binding of libfprefill (include/fprefill.h).

Argument marshalling only: tensors become device pointers, the varlen
descriptors stay host int32 arrays, and every computation runs in the CUDA
library.  PyTorch provides device memory and the current stream.  There is
no fallback: if the shared library has not been built, loading fails.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from ctypes import POINTER, Structure, c_float, c_int, c_longlong, c_size_t, c_uint64, c_void_p

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfprefill.so")

FP_OK, FP_ERR_INVALID, FP_ERR_UNSUPPORTED, FP_ERR_WORKSPACE, FP_ERR_CUDA, FP_ERR_DEVICE_BOUNDS, \
    FP_ERR_TIMEOUT = range(7)
FP_BF16, FP_E4M3 = 0, 1
FP_MAX_BATCH = 128
FP_SELECT_THRESHOLD, FP_SELECT_TOPK, FP_SELECT_TOPP = 0, 1, 2
FP_SCORE_PACKED, FP_SCORE_HEAD_UNION = 0, 1
FP_V_TOKEN_MAJOR, FP_V_DIM_MAJOR = 0, 1
FP_ROPE_HALF, FP_ROPE_INTERLEAVED = 0, 1
FP_WS_HEADER_BYTES = 256
FP_TABLES_MAX_BATCH = 4096


class FpParams(Structure):
    _fields_ = [("block", c_int), ("sink_tokens", c_int), ("local_tokens", c_int),
                ("alpha", c_float), ("softmax_scale", c_float), ("mean_correction", c_int),
                ("kv_splits", c_int), ("select_rule", c_int), ("top_k", c_int), ("top_p", c_float),
                ("score_mode", c_int), ("p_terms", c_int)]


class FpProblem(Structure):
    _fields_ = [("batch", c_int), ("h_q", c_int), ("h_kv", c_int), ("d", c_int), ("dtype", c_int),
                ("cu_seqlens_q", c_void_p), ("seqlens_k", c_void_p), ("q_start_pos", c_void_p),
                ("q", c_void_p), ("q_stride_tok", c_longlong), ("q_stride_head", c_longlong),
                ("k_cache", c_void_p), ("v_cache", c_void_p), ("page_size", c_int),
                ("num_pages", c_int), ("block_table", c_void_p), ("max_pages_per_seq", c_int),
                ("q_scale", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p), ("v_layout", c_int)]


class FpTables(Structure):
    _fields_ = [("batch", c_int), ("page_size", c_int), ("num_pages", c_int), ("max_pages_per_seq", c_int),
                ("num_free", c_int), ("capacity", c_int), ("seqlens", c_void_p), ("new_lens", c_void_p),
                ("free_pages", c_void_p), ("free_head", c_void_p), ("block_table", c_void_p),
                ("cu_seqlens_q", c_void_p), ("seqlens_k", c_void_p), ("positions", c_void_p), ("slots", c_void_p),
                ("free_next", c_void_p)]


class FpQCache(Structure):
    _fields_ = [("data", c_void_p), ("num_pages", c_int), ("page_size", c_int), ("h_kv", c_int), ("d", c_int),
                ("group", c_int)]


class FpQCacheRows(Structure):
    _fields_ = [("rows", c_int), ("dtype", c_int), ("k", c_void_p), ("v", c_void_p), ("stride_tok", c_longlong),
                ("stride_head", c_longlong), ("slots", c_void_p), ("out_slots", c_void_p), ("out_rows", c_int),
                ("k_scale", c_void_p), ("v_scale", c_void_p)]


class FpQCacheQuery(Structure):
    _fields_ = [("batch", c_int), ("h_q", c_int), ("total_q", c_int), ("max_q", c_int), ("dtype", c_int),
                ("q", c_void_p), ("q_stride_tok", c_longlong), ("q_stride_head", c_longlong), ("q_scale", c_void_p),
                ("cu_seqlens_q", c_void_p), ("seqlens_k", c_void_p), ("block_table", c_void_p),
                ("max_pages_per_seq", c_int), ("softmax_scale", c_float)]


class FpRopeTable(Structure):
    _fields_ = [("rot", c_int), ("layout", c_int), ("scale", c_float), ("turns", c_void_p)]


class FpRopeRows(Structure):
    _fields_ = [("rows", c_int), ("heads", c_int), ("x", c_void_p), ("x_stride_tok", c_longlong),
                ("x_stride_head", c_longlong), ("out", c_void_p), ("out_stride_tok", c_longlong),
                ("out_stride_head", c_longlong), ("out_dtype", c_int), ("out_scale", c_void_p), ("positions", c_void_p),
                ("inverse", c_int)]


class FpCache(Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("num_pages", c_int), ("page_size", c_int), ("h_kv", c_int),
                ("d", c_int), ("dtype", c_int), ("k_scale", c_void_p), ("v_scale", c_void_p)]


class FpCacheRows(Structure):
    _fields_ = [("rows", c_int), ("h_q", c_int), ("k", c_void_p), ("v", c_void_p), ("q", c_void_p),
                ("k_stride_tok", c_longlong), ("k_stride_head", c_longlong), ("v_stride_tok", c_longlong),
                ("v_stride_head", c_longlong), ("q_stride_tok", c_longlong), ("q_stride_head", c_longlong),
                ("q_out", c_void_p), ("q_out_stride_tok", c_longlong), ("q_out_stride_head", c_longlong),
                ("q_dtype", c_int), ("q_scale", c_void_p), ("slots", c_void_p), ("positions", c_void_p)]


# The same structures as bytes: packing them takes a fifth of the time of filling
# a ctypes one, which counts in calls of a few microseconds.
_PACK_TABLES = struct.Struct("@6i10P")
_PACK_ROWS = struct.Struct("@2i2P2q2Pi2P0P")
_PACK_QUERY = struct.Struct("@5iP2q4Pif0P")
_PACK_ROPE = struct.Struct("@2iP2qP2qi2Pi0P")
_PACK_APPEND = struct.Struct("@2i3P6qP2qi3P")
assert (_PACK_TABLES.size, _PACK_ROWS.size, _PACK_QUERY.size, _PACK_ROPE.size, _PACK_APPEND.size) == tuple(
    ctypes.sizeof(t) for t in (FpTables, FpQCacheRows, FpQCacheQuery, FpRopeRows, FpCacheRows))


class FprefillError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def lib():
    """The loaded shared library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libfprefill is not built ({_LIB_PATH} missing); "
                               "run block_sparse_long_fp_gb300.build.build()")
        L = ctypes.CDLL(_LIB_PATH)
        P, PP = POINTER(FpProblem), POINTER(FpParams)
        PT, PC, PR, PQ = POINTER(FpTables), POINTER(FpQCache), POINTER(FpQCacheRows), POINTER(FpQCacheQuery)
        sig = {
            "fp_default_params": ([], FpParams),
            "fp_num_rows": ([P, PP], c_longlong),
            "fp_num_key_blocks": ([P, PP], c_longlong),
            "fp_score_size": ([P, PP], c_longlong),
            "fp_total_q": ([P], c_longlong),
            "fp_score_offsets": ([P, PP, c_void_p, c_longlong], c_longlong),
            "fp_discover_workspace_size": ([P, PP], c_size_t),
            "fp_discover": ([P, PP, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p], c_int),
            "fp_select_workspace_size": ([P, PP], c_size_t),
            "fp_select": ([P, PP, c_void_p, c_void_p, c_void_p, c_longlong, c_void_p, c_void_p,
                           c_void_p, c_size_t, c_void_p], c_int),
            "fp_discover_select_workspace_size": ([P, PP], c_size_t),
            "fp_discover_select": ([P, PP, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_longlong, c_void_p,
                                    c_void_p, c_size_t, c_void_p], c_int),
            "fp_attn_workspace_size": ([P, PP], c_size_t),
            "fp_attn_kv_splits": ([P, PP], c_int),
            "fp_sparse_attn": ([P, PP, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_size_t, c_void_p], c_int),
            "fp_dense_attn": ([P, PP, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p], c_int),
            "fp_sparse_attn_noalloc": ([P, PP, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p], c_int),
            "fp_page_tables": ([PT, c_void_p, c_size_t, c_void_p], c_int),
            "fp_qcache_chunk_bytes": ([PC], c_size_t),
            "fp_qcache_bytes": ([PC], c_size_t),
            "fp_qcache_write": ([PC, PR, c_void_p, c_size_t, c_void_p], c_int),
            "fp_qcache_read": ([PC, PR, c_void_p, c_size_t, c_void_p], c_int),
            "fp_qcache_attn_scratch_bytes": ([PC, PQ], c_size_t),
            "fp_qcache_attn": ([PC, PQ, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_size_t, c_void_p], c_int),
            "fp_rope_turns": ([c_void_p, c_int, c_void_p], c_int),
            "fp_rope": ([POINTER(FpRopeTable), POINTER(FpRopeRows), c_void_p], c_int),
            "fp_cache_append": ([POINTER(FpCache), POINTER(FpRopeTable), POINTER(FpCacheRows), c_void_p, c_size_t,
                                 c_void_p], c_int),
            "fp_cache_attn_scratch_bytes": ([POINTER(FpCache), PQ], c_size_t),
            "fp_cache_attn": ([POINTER(FpCache), PQ, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_size_t, c_void_p],
                              c_int),
            "fp_reset_status": ([c_void_p, c_void_p], c_int),
            "fp_device_status": ([c_void_p, c_void_p, POINTER(c_int)], c_int),
            "fp_status_string": ([c_int], ctypes.c_char_p),
            "fp_set_wait_limit_ns": ([c_uint64], None),
            "fp_check_wait_timeout": ([c_void_p, c_uint64, c_void_p], c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().fp_status_string(int(s)).decode()


def _check(s: int, what: str):
    if s != FP_OK:
        raise FprefillError(s, what)


def default_params(**over) -> FpParams:
    p = lib().fp_default_params()
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream_handle(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


class Layer:
    """One attention layer's operands: device tensors (q, paged k/v caches,
    block table, FP8 scales) plus the host varlen descriptors.

    q: [total_q, h_q, 128] bf16 (or uint8 e4m3 codes); k_cache:
    [num_pages, page_size, h_kv, 128]; v_cache: the same, or
    [num_pages, h_kv, 128, page_size] with v_layout = FP_V_DIM_MAJOR;
    block_table: int32 [batch, max_pages].
    cu_seqlens_q / seqlens_k / q_start_pos: host int sequences.
    """

    def __init__(self, q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, q_start_pos,
                 h_q: int, h_kv: int, dtype: str = "bf16", q_scale=None, k_scale=None, v_scale=None,
                 params: FpParams | None = None, v_layout: int = 0):
        self.q, self.k_cache, self.v_cache, self.block_table = q, k_cache, v_cache, block_table
        self.q_scale, self.k_scale, self.v_scale = q_scale, k_scale, v_scale
        self.cu = np.ascontiguousarray(cu_seqlens_q, dtype=np.int32)
        self.lk = np.ascontiguousarray(seqlens_k, dtype=np.int32)
        self.start = np.ascontiguousarray(q_start_pos, dtype=np.int32)
        self.h_q, self.h_kv = h_q, h_kv
        self.params = params if params is not None else default_params()
        pr = FpProblem()
        pr.batch = len(self.lk)
        pr.h_q, pr.h_kv, pr.d = h_q, h_kv, int(q.shape[-1])
        pr.dtype = FP_BF16 if dtype == "bf16" else FP_E4M3
        pr.cu_seqlens_q = self.cu.ctypes.data
        pr.seqlens_k = self.lk.ctypes.data
        pr.q_start_pos = self.start.ctypes.data
        pr.q = _ptr(q)
        pr.q_stride_tok = int(q.stride(0))
        pr.q_stride_head = int(q.stride(1))
        pr.k_cache, pr.v_cache = _ptr(k_cache), _ptr(v_cache)
        pr.page_size = int(k_cache.shape[1])
        pr.num_pages = int(k_cache.shape[0])
        pr.block_table = _ptr(block_table)
        pr.max_pages_per_seq = int(block_table.shape[1])
        pr.q_scale, pr.k_scale, pr.v_scale = _ptr(q_scale), _ptr(k_scale), _ptr(v_scale)
        pr.v_layout = int(v_layout)
        self.problem = pr
        L = lib()
        pp, pm = ctypes.byref(pr), ctypes.byref(self.params)
        self.rows = int(L.fp_num_rows(pp, pm))
        if self.rows < 0:
            raise FprefillError(FP_ERR_INVALID, "varlen descriptors")
        self.key_blocks = int(L.fp_num_key_blocks(pp, pm))
        self.score_size = int(L.fp_score_size(pp, pm))
        self.total_q = int(L.fp_total_q(pp))
        self.kv_splits = int(L.fp_attn_kv_splits(pp, pm))   # split-KV parts of the attention calls
        self.ws_bytes = max(int(L.fp_discover_workspace_size(pp, pm)),
                            int(L.fp_select_workspace_size(pp, pm)),
                            int(L.fp_discover_select_workspace_size(pp, pm)),
                            int(L.fp_attn_workspace_size(pp, pm)))
        self._ws = None

    def score_offsets(self) -> np.ndarray:
        """fp_score_offsets: int64 [rows + 1], the start of every score-map row
        and, last, the map's size."""
        offs = np.zeros(self.rows + 1, dtype=np.int64)
        n = lib().fp_score_offsets(*self._refs(), offs.ctypes.data, offs.size)
        if n != offs.size:
            raise FprefillError(FP_ERR_INVALID, "fp_score_offsets")
        return offs

    # -- plumbing -------------------------------------------------------------
    def _refs(self):
        return ctypes.byref(self.problem), ctypes.byref(self.params)

    def workspace(self):
        import torch
        if self._ws is None:
            self._ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.q.device)
            _check(lib().fp_reset_status(_ptr(self._ws), _stream_handle()), "fp_reset_status")
        return self._ws

    def reset_status(self):
        _check(lib().fp_reset_status(_ptr(self.workspace()), _stream_handle()), "fp_reset_status")

    def check_wait_timeout(self, limit_ns: int):
        """fp_check_wait_timeout on this layer's workspace."""
        _check(lib().fp_check_wait_timeout(_ptr(self.workspace()), int(limit_ns), _stream_handle()),
               "fp_check_wait_timeout")

    def device_status(self) -> int:
        v = c_int(0)
        _check(lib().fp_device_status(_ptr(self.workspace()), _stream_handle(), ctypes.byref(v)),
               "fp_device_status")
        return v.value

    # -- the four stages ----------------------------------------------------------
    def discover(self, k_mean=None, v_mean=None, score=None):
        import torch
        dev = self.q.device
        shape = (self.key_blocks, self.h_kv, int(self.q.shape[-1]))
        k_mean = k_mean if k_mean is not None else torch.empty(shape, dtype=torch.float32, device=dev)
        v_mean = v_mean if v_mean is not None else torch.empty(shape, dtype=torch.float32, device=dev)
        score = score if score is not None else torch.empty(max(1, self.score_size), dtype=torch.float32,
                                                            device=dev)
        ws = self.workspace()
        _check(lib().fp_discover(*self._refs(), _ptr(k_mean), _ptr(v_mean), _ptr(score), _ptr(ws),
                                 self.ws_bytes, _stream_handle()), "fp_discover")
        return k_mean, v_mean, score

    def select(self, score, row_ptr=None, col_idx=None, nnz=None, dense_mask=None):
        import torch
        dev = self.q.device
        row_ptr = row_ptr if row_ptr is not None else torch.empty(self.rows + 1, dtype=torch.int32, device=dev)
        col_idx = col_idx if col_idx is not None else torch.empty(max(1, self.score_size), dtype=torch.int32,
                                                                  device=dev)
        nnz = nnz if nnz is not None else torch.empty(1, dtype=torch.int32, device=dev)
        ws = self.workspace()
        _check(lib().fp_select(*self._refs(), _ptr(score), _ptr(row_ptr), _ptr(col_idx), col_idx.numel(),
                               _ptr(nnz), _ptr(dense_mask), _ptr(ws), self.ws_bytes, _stream_handle()),
               "fp_select")
        return row_ptr, col_idx, nnz

    def discover_select(self, k_mean=None, v_mean=None, score=None, row_ptr=None, col_idx=None, nnz=None):
        """fp_discover_select: block means and the CSR index in one call (the
        score map only when `score` is given)."""
        import torch
        dev = self.q.device
        shape = (self.key_blocks, self.h_kv, int(self.q.shape[-1]))
        k_mean = k_mean if k_mean is not None else torch.empty(shape, dtype=torch.float32, device=dev)
        v_mean = v_mean if v_mean is not None else torch.empty(shape, dtype=torch.float32, device=dev)
        row_ptr = row_ptr if row_ptr is not None else torch.empty(self.rows + 1, dtype=torch.int32, device=dev)
        col_idx = col_idx if col_idx is not None else torch.empty(max(1, self.score_size), dtype=torch.int32,
                                                                  device=dev)
        nnz = nnz if nnz is not None else torch.empty(1, dtype=torch.int32, device=dev)
        ws = self.workspace()
        _check(lib().fp_discover_select(*self._refs(), _ptr(k_mean), _ptr(v_mean), _ptr(score), _ptr(row_ptr),
                                        _ptr(col_idx), col_idx.numel(), _ptr(nnz), _ptr(ws), self.ws_bytes,
                                        _stream_handle()), "fp_discover_select")
        return k_mean, v_mean, row_ptr, col_idx, nnz

    def _out(self, out, lse):
        import torch
        dev = self.q.device
        out = out if out is not None else torch.empty((self.total_q, self.h_q, int(self.q.shape[-1])),
                                                      dtype=torch.bfloat16, device=dev)
        return out, lse

    def sparse_attn(self, row_ptr, col_idx, k_mean, v_mean, out=None, lse=None, want_lse=True):
        import torch
        out, lse = self._out(out, lse)
        if lse is None and want_lse:
            lse = torch.empty((self.h_q, self.total_q), dtype=torch.float32, device=self.q.device)
        ws = self.workspace()
        _check(lib().fp_sparse_attn(*self._refs(), _ptr(row_ptr), _ptr(col_idx), _ptr(k_mean), _ptr(v_mean),
                                    _ptr(out), _ptr(lse), _ptr(ws), self.ws_bytes, _stream_handle()),
               "fp_sparse_attn")
        return out, lse

    def sparse_attn_noalloc(self, row_ptr, col_idx, k_mean, v_mean, out, lse=None, status=None):
        """fp_sparse_attn_noalloc: same result as sparse_attn, with the
        library's built-in scratch instead of a workspace (nothing is
        allocated here either: out, lse and status are the caller's)."""
        _check(lib().fp_sparse_attn_noalloc(*self._refs(), _ptr(row_ptr), _ptr(col_idx), _ptr(k_mean),
                                            _ptr(v_mean), _ptr(out), _ptr(lse), _ptr(status),
                                            _stream_handle()), "fp_sparse_attn_noalloc")
        return out, lse

    def dense_attn(self, out=None, lse=None, want_lse=True):
        import torch
        out, lse = self._out(out, lse)
        if lse is None and want_lse:
            lse = torch.empty((self.h_q, self.total_q), dtype=torch.float32, device=self.q.device)
        ws = self.workspace()
        _check(lib().fp_dense_attn(*self._refs(), _ptr(out), _ptr(lse), _ptr(ws), self.ws_bytes,
                                   _stream_handle()), "fp_dense_attn")
        return out, lse

    def prefill(self, out=None, lse=None, want_lse=False):
        """One pass of the whole path: discover -> select -> sparse attention."""
        k_mean, v_mean, score = self.discover()
        row_ptr, col_idx, nnz = self.select(score)
        out, lse = self.sparse_attn(row_ptr, col_idx, k_mean, v_mean, out=out, lse=lse, want_lse=want_lse)
        return out, lse, (row_ptr, col_idx, nnz)


def _need(t, name: str, dtypes, device: int, ndim: int, contiguous: bool = True):
    """An argument check of the classes below: FprefillError (invalid argument) names the tensor."""
    if t.dtype in dtypes and t.dim() == ndim and t.get_device() == device and (not contiguous or t.is_contiguous()):
        return
    raise FprefillError(FP_ERR_INVALID, f"{name}: {ndim}-d {'contiguous ' if contiguous else ''}tensor of "
                        f"{' or '.join(str(d) for d in dtypes)} on cuda:{device} wanted, got {tuple(t.shape)} {t.dtype} "
                        f"on {t.device}")


class _OnDevice:
    """What PageTables, QCache, Rope and KVCache share: the status header, and calls on their
    device's current stream whatever device is current."""

    def __init__(self, device):
        import torch
        if device.type != "cuda":
            raise FprefillError(FP_ERR_INVALID, f"a CUDA tensor is wanted, got {device}")
        self._lib = lib()
        self._torch = torch
        self.device = device
        self._index = device.index
        self._ws = torch.zeros(FP_WS_HEADER_BYTES // 4, dtype=torch.int32, device=device)
        self._ws_ptr = self._ws.data_ptr()
        self._bf16, self._fp8 = (torch.bfloat16,), (torch.uint8, torch.float8_e4m3fn)
        self._int32, self._fp32 = torch.int32, torch.float32
        # the current stream's handle: the short way, where torch has it, saves a microsecond a call
        self._stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                               lambda index: torch.cuda.current_stream(index).cuda_stream)

    def _settle(self):
        """Waits for what the constructor enqueued, the status' zeros too: any stream may use the object from
        here on.  One built in a graph's capture is ready where the graph has run."""
        torch = self._torch
        with torch.cuda.device(self.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _entry(self, name: str, arguments: int):
        """An entry point that takes its structures as bytes, and integers."""
        f = self._lib._FuncPtr((name, self._lib))
        f.argtypes, f.restype = [c_void_p] * arguments, c_int
        return f

    def _call(self, f, what: str, *args):
        """The entry point f on the current stream of this object's device."""
        index = self._index
        if self._torch.cuda.current_device() == index:
            s = f(*args, self._stream(index))
        else:
            with self._torch.cuda.device(index):
                s = f(*args, self._stream(index))
        if s != FP_OK:
            raise FprefillError(s, what)

    def _vector(self, t, name: str, n: int) -> int:
        """The address of an int32 vector of n entries."""
        if t.dtype is self._int32 and t.shape == (n,) and t.get_device() == self._index and t.is_contiguous():
            return t.data_ptr()
        _need(t, name, (self._int32,), self._index, 1)
        raise FprefillError(FP_ERR_INVALID, f"{name}: {n} entries wanted, got {t.shape[0]}")

    def _scales(self, t, name: str, n: int) -> int:
        """The address of n fp32 scales."""
        if t is None:
            raise FprefillError(FP_ERR_INVALID, f"{name} is missing")
        if t.dtype is self._fp32 and t.shape == (n,) and t.get_device() == self._index and t.is_contiguous():
            return t.data_ptr()
        _need(t, name, (self._fp32,), self._index, 1)
        raise FprefillError(FP_ERR_INVALID, f"{name}: {n} entries wanted, got {t.shape[0]}")

    def _heads(self, t, name: str, heads, fp8: bool = False):
        """Address and strides of rows [rows, heads, 128] with contiguous dims (any number of heads when None)."""
        shape, strides = t.shape, t.stride()
        if not (len(shape) == 3 and t.dtype in (self._fp8 if fp8 else self._bf16) and t.get_device() == self._index and
                strides[2] == 1 and shape[2] == 128 and shape[1] and (heads is None or shape[1] == heads)):
            _need(t, name, self._fp8 if fp8 else self._bf16, self._index, 3, False)
            raise FprefillError(FP_ERR_INVALID, f"{name}: [rows, {'heads' if heads is None else heads}, 128] with contiguous "
                                f"dims wanted, got {tuple(shape)} {strides}")
        # a single row (or head) may carry any stride: the packed one stands for it
        stride_head = strides[1] if shape[1] > 1 else 128
        return t.data_ptr(), strides[0] if shape[0] > 1 else shape[1] * stride_head, stride_head

    def device_status(self) -> int:
        """Waits for the current stream; what its kernels found wrong in device data (FP_OK: nothing)."""
        v = c_int(0)
        with self._torch.cuda.device(self.device):
            _check(lib().fp_device_status(self._ws_ptr, _stream_handle(), ctypes.byref(v)), "fp_device_status")
        return v.value

    def reset_status(self):
        self._call(self._lib.fp_reset_status, "fp_reset_status", self._ws_ptr)


class PageTables(_OnDevice):
    """fp_page_tables: the block table, lengths and slot maps of a batch, step
    by step, on the GPU.

    block_table: int32 [batch, max_pages_per_seq], the caller's, updated in
    place.  The results -- cu_seqlens_q, seqlens_k, positions, slots,
    free_head, as fprefill.h describes them -- are buffers of this object that
    each step overwrites: calls that overlap on the GPU need one object each.
    """

    def __init__(self, block_table, page_size: int, num_pages: int, capacity: int):
        import torch
        super().__init__(block_table.device)
        _need(block_table, "block_table", (torch.int32,), self._index, 2)
        if capacity < 1:
            raise FprefillError(FP_ERR_INVALID, "capacity")
        self.block_table, self.capacity = block_table, int(capacity)
        batch = block_table.shape[0]

        def new(n):
            return torch.empty(n, dtype=torch.int32, device=self.device)
        self.cu_seqlens_q, self.seqlens_k, self.free_head = new(batch + 1), new(batch), new(1)
        self.positions, self.slots = new(self.capacity), new(self.capacity)
        t = self._t = FpTables()
        t.batch, t.max_pages_per_seq = batch, block_table.shape[1]
        t.page_size, t.num_pages, t.capacity = int(page_size), int(num_pages), self.capacity
        t.block_table, t.cu_seqlens_q = _ptr(block_table), _ptr(self.cu_seqlens_q)
        t.seqlens_k, t.positions = _ptr(self.seqlens_k), _ptr(self.positions)
        t.slots, t.free_next = _ptr(self.slots), _ptr(self.free_head)
        self._shape = (t.batch, t.page_size, t.num_pages, t.max_pages_per_seq)
        self._out = (t.block_table, t.cu_seqlens_q, t.seqlens_k, t.positions, t.slots, t.free_next)
        self._f = self._entry("fp_page_tables", 4)

    def step(self, seqlens, new_lens, free_pages, free_head=None):
        """One step (returns this object).  seqlens, new_lens: int32 [batch];
        free_pages: int32, used from entry free_head (int32 [1], 0 when None)
        on.  Passing this object's own seqlens_k and free_head advances both in
        place."""
        batch, free = self._shape[0], free_pages.shape[0]
        t = _PACK_TABLES.pack(*self._shape, free, self.capacity, self._vector(seqlens, "seqlens", batch),
                              self._vector(new_lens, "new_lens", batch), self._vector(free_pages, "free_pages", free),
                              0 if free_head is None else self._vector(free_head, "free_head", 1), *self._out)
        self._call(self._f, "fp_page_tables", t, self._ws_ptr, FP_WS_HEADER_BYTES)
        return self


class _Scratch:
    """Memory of one stream, and the lock of those who enqueue calls that use it."""

    def __init__(self):
        self.memory, self.lock = None, threading.Lock()


class _Cache(_OnDevice):
    """What QCache and KVCache share: attention over their pages, and its scratch."""

    _scratch = {}              # _Scratch by device and stream, for all objects: a model's layers run one behind the other

    def _entries(self, attn: str, *others):
        """Sets up the entry points: `others`, pairs of names and argument counts, and last the attention's."""
        self._scratch_bytes = {}
        self._f = tuple(self._entry(*f) for f in others) + (self._entry(attn, 9),)
        self._attn_name, self._scratch_query = attn, getattr(self._lib, attn + "_scratch_bytes")
        self._settle()

    def attn(self, q, block_table, seqlens_k, cu_seqlens_q=None, max_q=None, out=None, lse=None, want_lse=True,
             q_scale=None, softmax_scale: float = 0.0):
        """Attention of q (bf16 [total_q, h_q, 128], or e4m3 with q_scale [h_q])
        over the cached tokens: (out bf16 [total_q, h_q, 128], lse fp32 [h_q,
        total_q] or None).

        block_table int32 [batch, max_pages], seqlens_k int32 [batch] (the
        queries' own tokens included).  Request r owns rows cu_seqlens_q[r] ..
        cu_seqlens_q[r+1]-1 (int32 [batch+1]), at most max_q; without
        cu_seqlens_q, max_q rows each (by default total_q / batch, which has to
        be a whole number).  Rows behind the last request's are not written:
        in an `out` of this call's own they are what the memory held."""
        torch, dev, h_kv = self._torch, self._index, self.h_kv
        shape, strides = q.shape, q.stride()
        kinds = self._bf16 if q_scale is None else self._fp8
        if not (len(shape) == 3 and q.dtype in kinds and q.get_device() == dev and strides[2] == 1 and shape[2] == 128 and
                shape[1] % h_kv == 0):
            _need(q, "q", kinds, dev, 3, False)
            raise FprefillError(FP_ERR_INVALID, f"q: [rows, a multiple of {h_kv}, 128] with contiguous dims wanted, "
                                f"got {tuple(shape)} {strides}")
        total_q, h_q, _ = shape
        batch = seqlens_k.shape[0]
        seqlens_at = self._vector(seqlens_k, "seqlens_k", batch)
        if not (block_table.dtype is self._int32 and block_table.dim() == 2 and block_table.shape[0] == batch and
                block_table.get_device() == dev and block_table.is_contiguous()):
            _need(block_table, "block_table", (self._int32,), dev, 2)
            raise FprefillError(FP_ERR_INVALID, f"block_table: {batch} rows wanted, one for each length")
        width = block_table.shape[1]
        cu_at = 0 if cu_seqlens_q is None else self._vector(cu_seqlens_q, "cu_seqlens_q", batch + 1)
        if max_q is None:
            if cu_seqlens_q is None and batch and total_q % batch:
                raise FprefillError(FP_ERR_INVALID, f"{total_q} rows are no equal share of {batch} requests: cu_seqlens_q or "
                                    "max_q wanted")
            max_q = max(1, total_q // batch if batch and cu_seqlens_q is None else total_q)
        stride_head = strides[1] if h_q > 1 else 128
        Q = _PACK_QUERY.pack(batch, h_q, total_q, max_q, FP_BF16 if q_scale is None else FP_E4M3, q.data_ptr(),
                             strides[0] if total_q > 1 else h_q * stride_head, stride_head,
                             0 if q_scale is None else self._scales(q_scale, "q_scale", h_q), cu_at, seqlens_at,
                             block_table.data_ptr(), width, softmax_scale)
        if out is None:
            out = torch.empty((total_q, h_q, 128), dtype=torch.bfloat16, device=self.device)
        elif out.shape != shape or out.dtype is not torch.bfloat16 or out.get_device() != dev or not out.is_contiguous():
            _need(out, "out", self._bf16, dev, 3)
            raise FprefillError(FP_ERR_INVALID, "out: the shape of q wanted")
        if lse is not None:
            _need(lse, "lse", (self._fp32,), dev, 2)
            if lse.shape != (h_q, total_q):
                raise FprefillError(FP_ERR_INVALID, "lse: [h_q, total_q] wanted")
        elif want_lse:
            lse = torch.empty((h_q, total_q), dtype=self._fp32, device=self.device)
        key = (batch, h_q, total_q, max_q, cu_at == 0, width, q_scale is None)
        n = self._scratch_bytes.get(key)
        if n is None:
            if len(self._scratch_bytes) >= 512:        # a server's rows may take any number of shapes
                self._scratch_bytes.clear()
            n = self._scratch_bytes[key] = int(
                self._scratch_query(self._c, FpQCacheQuery.from_buffer_copy(Q)))
        args = (self._bytes, Q, out.data_ptr(), 0 if lse is None else lse.data_ptr())
        if torch.cuda.current_device() == dev:
            self._attn(args, n)
        else:
            with torch.cuda.device(dev):
                self._attn(args, n)
        return out, lse

    def _attn(self, args, n: int):
        """The attention with n bytes of scratch of the current stream, which holds nothing between calls: calls on
        two streams share none, and a captured call has its own, out of the graph's memory.  The library enqueues
        several kernels that hand partial results over in it: of threads on one stream, one enqueues at a time."""
        torch, stream = self._torch, self._stream(self._index)
        mine = self._scratch.get((self._index, stream))
        if mine is None:
            mine = self._scratch.setdefault((self._index, stream), _Scratch())       # one of two threads' stays
        capturing = torch.cuda.is_current_stream_capturing()
        with mine.lock:
            scratch = None if capturing else mine.memory
            if scratch is None or scratch.numel() < n:
                scratch = torch.empty(max(16, n), dtype=torch.uint8, device=self.device)
                if not capturing:
                    mine.memory = scratch
            s = self._f[-1](*args, scratch.data_ptr(), n, self._ws_ptr, FP_WS_HEADER_BYTES, stream)
        if s != FP_OK:
            raise FprefillError(s, self._attn_name)


class QCache(_Cache):
    """A paged K/V cache held in 4 bits: fp_qcache_write, fp_qcache_read and
    fp_qcache_attn on it.

    data: uint8 [num_pages, h_kv, page_size / 16, chunk_bytes] in the layout
    that fprefill.h documents (QCache.empty makes one).  e4m3 tensors are uint8
    codes or torch.float8_e4m3fn.
    """

    def __init__(self, data, page_size: int, group: int = 32):
        import torch
        super().__init__(data.device)
        _need(data, "data", (torch.uint8,), self._index, 4)
        c = self._c = FpQCache()
        c.data, c.num_pages, c.h_kv, c.d = _ptr(data), data.shape[0], data.shape[1], 128
        c.page_size, c.group = int(page_size), int(group)
        if not int(lib().fp_qcache_bytes(c)):
            raise FprefillError(FP_ERR_UNSUPPORTED, f"a 4-bit cache with pages of {page_size}, groups of {group}")
        if data.numel() != int(lib().fp_qcache_bytes(c)) or data.shape[2] * 16 != c.page_size:
            raise FprefillError(FP_ERR_INVALID, f"data: [pages, heads, {c.page_size // 16}, {self.chunk_bytes(group)}] "
                                f"wanted, got {tuple(data.shape)}")
        self.data, self.h_kv, self.page_size, self.group = data, c.h_kv, c.page_size, c.group
        self._bytes = bytes(c)
        self._entries("fp_qcache_attn", ("fp_qcache_write", 5), ("fp_qcache_read", 5))

    @staticmethod
    def chunk_bytes(group: int = 32) -> int:
        return 2048 + 128 * (128 // group)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, h_kv: int, group: int = 32, device="cuda"):
        """An uninitialised cache."""
        import torch
        if group not in (32, 64, 128):
            raise FprefillError(FP_ERR_UNSUPPORTED, f"groups of {group}")
        return cls(torch.empty((num_pages, h_kv, page_size // 16, cls.chunk_bytes(group)), dtype=torch.uint8,
                               device=device), page_size, group)

    def _rows(self, k, v, slots, k_scale, v_scale, out_slots=None):
        dev, h = self._index, self.h_kv
        fp8 = k_scale is not None or v_scale is not None
        kinds = self._fp8 if fp8 else self._bf16
        shape, strides = k.shape, k.stride()
        if not (len(shape) == 3 and v.shape == shape and v.stride() == strides and shape[1] == h and shape[2] == 128 and
                strides[2] == 1 and k.dtype in kinds and v.dtype in kinds and k.get_device() == dev and
                v.get_device() == dev):
            _need(k, "k", kinds, dev, 3, False)
            _need(v, "v", kinds, dev, 3, False)
            raise FprefillError(FP_ERR_INVALID, f"k, v: [rows, {h}, 128] with like strides and contiguous dims wanted, "
                                f"got {tuple(shape)} {strides} and {tuple(v.shape)} {v.stride()}")
        rows = shape[0]
        n = rows if out_slots is None else slots.shape[0]
        slots_at = self._vector(slots, "slots", n)
        out_at = 0 if out_slots is None else self._vector(out_slots, "out_slots", n)
        # a single row (or head) may carry any stride: the packed one stands for it
        stride_head = strides[1] if h > 1 else 128
        return _PACK_ROWS.pack(n, FP_E4M3 if fp8 else FP_BF16, k.data_ptr(), v.data_ptr(),
                               strides[0] if rows > 1 else h * stride_head, stride_head, slots_at, out_at, rows,
                               self._scales(k_scale, "k_scale", h) if fp8 else 0,
                               self._scales(v_scale, "v_scale", h) if fp8 else 0)

    def write(self, k, v, slots, k_scale=None, v_scale=None):
        """Quantise rows of k and v (bf16 [rows, h_kv, 128], or e4m3 with one
        scale per head; k and v of like strides) into `slots` (int32 [rows];
        -1: none; none twice)."""
        self._call(self._f[0], "fp_qcache_write", self._bytes, self._rows(k, v, slots, k_scale, v_scale), self._ws_ptr, FP_WS_HEADER_BYTES)

    def read(self, slots, k_out=None, v_out=None, out_slots=None, k_scale=None, v_scale=None):
        """Bring the tokens at `slots` back into k_out and v_out (bf16 [.., h_kv,
        128], or e4m3 with one scale per head): row i, or row out_slots[i].
        Without k_out and v_out, new bf16 rows, zero where a slot is -1.  A
        paged cache is passed as its rows: k_cache.flatten(0, 1)."""
        if (k_out is None) != (v_out is None):
            raise FprefillError(FP_ERR_INVALID, "k_out and v_out come together")
        if k_out is None:
            if out_slots is not None or k_scale is not None:
                raise FprefillError(FP_ERR_INVALID, "out_slots and e4m3 want k_out and v_out")
            torch = self._torch
            k_out, v_out = (torch.zeros((slots.shape[0], self.h_kv, 128), dtype=torch.bfloat16, device=self.device)
                            for _ in range(2))
        self._call(self._f[1], "fp_qcache_read", self._bytes, self._rows(k_out, v_out, slots, k_scale, v_scale, out_slots),
                   self._ws_ptr, FP_WS_HEADER_BYTES)
        return k_out, v_out


def rope_frequencies(rot: int = 128, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int = 4096, low: float | None = None, high: float | None = None) -> np.ndarray:
    """Radians a position for the rot / 2 pairs of a rotary embedding, float64:
    base^(-2 i / rot), scaled for contexts `factor` times the trained ones by

    None       nothing;
    "linear"   1 / factor for every pair (positions squeezed);
    "base"     the base raised to base * factor^(rot / (rot - 2)), so that the
               longest wave is `factor` times as long and the shortest stays;
    "smooth"   by the waves that a pair makes in `original` positions: 1 / factor
               up to `low` waves (1), 1 from `high` (4) on, and linear in them between;
    "ramp"     the same, but linear in the pair's index between those indices
               (rounded outwards) where a pair makes `high` (32) and `low` (1)
               waves.  Models with a ramp mostly scale cos and sin as well:
               Rope(..., scale=0.1 * math.log(factor) + 1)."""
    low = 1.0 if low is None else low
    high = (32.0 if scaling == "ramp" else 4.0) if high is None else high
    if rot < 2 or rot > 128 or rot % 2 or not base > 1 or not factor > 0:
        raise FprefillError(FP_ERR_INVALID, f"rope_frequencies: rot {rot}, base {base}, factor {factor}")
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        if rot == 2:
            raise FprefillError(FP_ERR_INVALID, "rope_frequencies: one pair has no base to raise")
        return (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
    f = base ** (-2 * i / rot)
    if scaling is None:
        return f
    if scaling == "linear":
        return f / factor
    if scaling not in ("smooth", "ramp") or not original > 0 or not high > low > 0:
        raise FprefillError(FP_ERR_INVALID, f"rope_frequencies: scaling {scaling!r}, original {original}, low {low}, high {high}")
    if scaling == "smooth":
        keep = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0, 1)
    else:
        first, last = (rot * np.log(original / (w * 2 * np.pi)) / (2 * np.log(base)) for w in (high, low))
        first, last = max(0, np.floor(first)), min(rot - 1, np.ceil(last))
        keep = 1 - np.clip((i - first) / max(last - first, 0.001), 0, 1)
    return f * keep + f / factor * (1 - keep)


class Rope(_OnDevice):
    """Rotary positions: fp_rope, and the rotation that KVCache.append applies.

    inv_freq: rot / 2 frequencies in radians a position (rope_frequencies, or a
    model's own), for the first rot dims of a head; layout: "half" (pairs i, i +
    rot / 2) or "interleaved" (2 i, 2 i + 1); scale multiplies cos and sin.
    """

    def __init__(self, inv_freq, layout: str = "half", scale: float = 1.0, device="cuda"):
        import torch
        freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
        if freq.ndim != 1 or not 1 <= freq.size <= 64 or layout not in ("half", "interleaved") or not np.isfinite(scale):
            raise FprefillError(FP_ERR_INVALID, f"Rope: 1 to 64 frequencies, layout half or interleaved, a finite scale "
                                f"wanted, got {freq.shape}, {layout!r}, {scale}")
        turns = np.zeros(freq.size, dtype=np.uint64)
        _check(lib().fp_rope_turns(freq.ctypes.data, freq.size, turns.ctypes.data), "fp_rope_turns")
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        super().__init__(self.turns.device)
        self._settle()
        self.rot, self.layout, self.scale = 2 * freq.size, layout, float(scale)
        self._t = FpRopeTable(self.rot, FP_ROPE_INTERLEAVED if layout == "interleaved" else FP_ROPE_HALF, self.scale,
                              _ptr(self.turns))
        self._bytes = bytes(self._t)
        self._f = self._entry("fp_rope", 3)

    def apply(self, x, positions, out=None, out_scale=None, inverse: bool = False):
        """x (bf16 [rows, heads, 128]) rotated by positions (int32 [rows]); with
        inverse, back (the gradient's rotation too).  Into out -- bf16, x itself
        if wanted, or with out_scale [heads] e4m3 -- or into new rows.  As with
        every call here, the result has no history: a backward pass calls it
        with inverse itself."""
        x_at = self._heads(x, "x", None)
        rows, heads = x.shape[0], x.shape[1]
        fp8 = out_scale is not None
        if out is None:
            out = self._torch.empty((rows, heads, 128), dtype=self._torch.uint8 if fp8 else self._torch.bfloat16,
                                    device=self.device)
        out_at = self._heads(out, "out", heads, fp8)
        if out.shape[0] != rows:
            raise FprefillError(FP_ERR_INVALID, f"out: {rows} rows wanted, got {out.shape[0]}")
        R = _PACK_ROPE.pack(rows, heads, *x_at, *out_at, FP_E4M3 if fp8 else FP_BF16,
                            self._scales(out_scale, "out_scale", heads) if fp8 else 0,
                            self._vector(positions, "positions", rows), 1 if inverse else 0)
        self._call(self._f, "fp_rope", self._bytes, R)
        return out


class KVCache(_Cache):
    """The bf16 or e4m3 paged K/V cache that Layer reads, at any position:
    fp_cache_append and fp_cache_attn on it.

    k_cache, v_cache: [num_pages, page_size, h_kv, 128], bf16, or e4m3 (uint8
    codes or torch.float8_e4m3fn) with k_scale and v_scale (fp32 [h_kv]).  Layer's
    value caches by columns (v_layout 1) are not read here.
    """

    def __init__(self, k_cache, v_cache, k_scale=None, v_scale=None):
        super().__init__(k_cache.device)
        fp8 = k_scale is not None or v_scale is not None
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, name, self._fp8 if fp8 else self._bf16, self._index, 4)
        if v_cache.shape != k_cache.shape or k_cache.shape[3] != 128:
            raise FprefillError(FP_ERR_INVALID, f"k_cache, v_cache: [num_pages, page_size, h_kv, 128] wanted, got "
                                f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
        c = self._c = FpCache()
        c.k, c.v, c.d, c.dtype = _ptr(k_cache), _ptr(v_cache), 128, FP_E4M3 if fp8 else FP_BF16
        c.num_pages, c.page_size, c.h_kv = (int(n) for n in k_cache.shape[:3])
        if c.page_size < 16 or (128 % c.page_size and c.page_size % 128):
            raise FprefillError(FP_ERR_UNSUPPORTED, f"pages of {c.page_size} tokens")
        if fp8:
            c.k_scale, c.v_scale = (self._scales(t, n, c.h_kv) for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")))
        self.k_cache, self.v_cache, self.k_scale, self.v_scale = k_cache, v_cache, k_scale, v_scale
        self.h_kv, self.page_size = c.h_kv, c.page_size
        self._bytes = bytes(c)
        self._entries("fp_cache_attn", ("fp_cache_append", 6))

    def append(self, k, v, slots, rope: Rope | None = None, positions=None, q=None, q_out=None, q_scale=None):
        """Rows of k and v (bf16 [rows, h_kv, 128]) into `slots` (int32 [rows]; -1:
        none; none twice).  With a Rope, k and q rotated by positions (int32
        [rows]).  Returns q (bf16 [rows, h_q, 128]) so rotated, in q_out -- bf16,
        q itself if wanted, or with q_scale [h_q] e4m3 -- or in new rows; None
        without q."""
        k_at, v_at = self._heads(k, "k", self.h_kv), self._heads(v, "v", self.h_kv)
        rows = k.shape[0]
        if v.shape[0] != rows:
            raise FprefillError(FP_ERR_INVALID, f"v: {rows} rows wanted, got {v.shape[0]}")
        slots_at = self._vector(slots, "slots", rows)
        if (rope is None) != (positions is None):
            raise FprefillError(FP_ERR_INVALID, "rope and positions come together")
        if rope is not None and rope._index != self._index:
            raise FprefillError(FP_ERR_INVALID, f"rope: on cuda:{self._index} wanted, got {rope.device}")
        q_at, out_at, h_q, scale_at = (0, 0, 0), (0, 0, 0), 0, 0
        if q is not None:
            q_at = self._heads(q, "q", None)
            h_q = q.shape[1]
            fp8 = q_scale is not None
            if q_out is None:
                q_out = self._torch.empty((rows, h_q, 128), dtype=self._torch.uint8 if fp8 else self._torch.bfloat16,
                                          device=self.device)
            out_at = self._heads(q_out, "q_out", h_q, fp8)
            if q.shape[0] != rows or q_out.shape[0] != rows:
                raise FprefillError(FP_ERR_INVALID, f"q, q_out: {rows} rows wanted, got {q.shape[0]}, {q_out.shape[0]}")
            if fp8:
                scale_at = self._scales(q_scale, "q_scale", h_q)
        elif q_out is not None or q_scale is not None:
            raise FprefillError(FP_ERR_INVALID, "q_out and q_scale want q")
        # an empty batch may have no memory: a q of no rows is no q
        R = _PACK_APPEND.pack(rows, h_q if q_at[0] else 0, k_at[0], v_at[0], q_at[0], *k_at[1:], *v_at[1:], *q_at[1:],
                              *out_at, FP_E4M3 if scale_at else FP_BF16, scale_at, slots_at,
                              0 if rope is None else self._vector(positions, "positions", rows))
        self._call(self._f[0], "fp_cache_append", self._bytes, 0 if rope is None else rope._bytes, R, self._ws_ptr,
                   FP_WS_HEADER_BYTES)
        return q_out


def layer_from_case(case, device="cuda", params: FpParams | None = None, v_layout: int = 0):
    """Upload a synthetic case (block_sparse_long_fp_gb300.synth.Case) and wrap it.
    v_layout = FP_V_DIM_MAJOR uploads the value cache as [num_pages, h_kv, 128,
    page_size] (the same values, keys contiguous)."""
    import torch
    spec = case.spec
    v_host = case.v_cache if v_layout == FP_V_TOKEN_MAJOR else np.ascontiguousarray(case.v_cache.transpose(0, 2, 3, 1))
    if spec.dtype == "bf16":
        q = torch.from_numpy(case.q).view(torch.bfloat16).to(device)
        k = torch.from_numpy(case.k_cache).view(torch.bfloat16).to(device)
        v = torch.from_numpy(v_host).view(torch.bfloat16).to(device)
        qs = ks = vs = None
    else:
        q = torch.from_numpy(case.q).to(device)
        k = torch.from_numpy(case.k_cache).to(device)
        v = torch.from_numpy(v_host).to(device)
        qs = torch.from_numpy(case.q_scale).to(device)
        ks = torch.from_numpy(case.k_scale).to(device)
        vs = torch.from_numpy(case.v_scale).to(device)
    bt = torch.from_numpy(case.block_table).to(device)
    return Layer(q, k, v, bt, case.cu_seqlens_q, case.seqlens_k, case.q_start_pos, spec.h_q, spec.h_kv,
                 dtype=spec.dtype, q_scale=qs, k_scale=ks, v_scale=vs, params=params, v_layout=v_layout)

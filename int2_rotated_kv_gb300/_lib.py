"""ctypes binding of liboscar.so (include/oscar.h).  Argument marshalling only:
every step of the path runs in the library.  The functions keep the C names.

Device arguments are torch CUDA tensors (PyTorch is used for device memory and
streams); host-side calls take numpy arrays.  A missing library raises at
import time -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "liboscar.so")

OSCAR_OK = 0
STATUS_NAMES = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED", -3: "WORKSPACE", -4: "CUDA",
                -5: "NOT_CONVERGED"}
DEVERR_PAGE_ID, DEVERR_TIMEOUT, DEVERR_SEQ_LEN, DEVERR_NONFINITE = 1, 2, 4, 8
DEVERR_NO_PAGES = 16
KV8_INT8, KV8_E4M3 = 0, 1
VARIANT_OSCAR, VARIANT_HADAMARD, VARIANT_IDENTITY = 0, 1, 2
EXPORTED = ("oscar_query_covariance", "oscar_score_covariance", "oscar_build_rotation",
            "oscar_prefill_quantize", "oscar_quantize_append", "oscar_decode_workspace_size",
            "oscar_decode_attention", "oscar_decode_attention_bf16", "oscar_device_sm_count",
            "oscar_status_string", "oscar_version", "oscar_decode_attention_static",
            "oscar_decode_step", "oscar_decode_step_rope", "oscar_multiquery_attention",
            "oscar_multiquery_workspace_size", "oscar_decode_step_host_staging_size",
            "oscar_decode_step_host",
            "oscar_calibration_workspace_size", "oscar_query_covariance_device",
            "oscar_score_covariance_device", "oscar_clip_threshold_device",
            "oscar_prefill_quantize_trace", "oscar_quantize_append_trace",
            "oscar_kv8_place", "oscar_kv8_gather", "oscar_kv8_workspace_size",
            "oscar_kv8_attention", "oscar_kv4_place", "oscar_kv4_gather", "oscar_kv4_workspace_size",
            "oscar_kv4_attention", "oscar_gather", "oscar_extend_pages", "oscar_rope_phases", "oscar_rope")


class OscarError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {status} ({STATUS_NAMES.get(status, '?')}: "
                         f"{lib().oscar_status_string(status).decode()})")


class CacheDesc(ctypes.Structure):
    _fields_ = [
        ("num_kv_heads", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("sink", ctypes.c_int32), ("window", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_int2_pages", ctypes.c_int64), ("num_bf16_pages", ctypes.c_int64),
        ("int2_pool", ctypes.c_void_p), ("bf16_pool", ctypes.c_void_p),
        ("int2_page_table", ctypes.c_void_p), ("bf16_page_table", ctypes.c_void_p),
        ("r_k", ctypes.c_void_p), ("r_v", ctypes.c_void_p),
        ("clip_k", ctypes.c_void_p), ("clip_v", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("code_bits", ctypes.c_int32),
    ]


class Kv4Desc(ctypes.Structure):
    _fields_ = [
        ("num_kv_heads", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int64), ("num_tails", ctypes.c_int64),
        ("pool", ctypes.c_void_p), ("tail", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("tail_ids", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


class Kv8Desc(ctypes.Structure):
    _fields_ = Kv4Desc._fields_ + [("format", ctypes.c_int32)]


_LIB = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m int2_rotated_kv_gb300.build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
        sig = {
            "oscar_query_covariance": (I32, [I32, I32, I64, P, P]),
            "oscar_score_covariance": (I32, [I32, I32, I64, P, P, P, I32, P]),
            "oscar_build_rotation": (I32, [I32, P, P, I64, D, I32, P, P, P, P]),
            "oscar_prefill_quantize": (I32, [P, P, P, P, P, P, I32, I64, P]),
            "oscar_quantize_append": (I32, [P, P, P, P, I32, P]),
            "oscar_prefill_quantize_trace": (I32, [P, P, P, P, P, P, I32, I64, P, P]),
            "oscar_quantize_append_trace": (I32, [P, P, P, P, I32, P, P]),
            "oscar_decode_workspace_size": (ctypes.c_size_t, [P, I32, I32]),
            "oscar_multiquery_workspace_size": (ctypes.c_size_t, [P, I32, I32, I32]),
            "oscar_decode_attention": (I32, [P, P, P, I32, I32, P, P, ctypes.c_size_t, P]),
            "oscar_decode_attention_bf16": (I32, [P, P, P, I32, I32, P, P, ctypes.c_size_t, P]),
            "oscar_device_sm_count": (I32, []),
            "oscar_decode_attention_static": (I32, [P, P, P, I32, I32, P, P]),
            "oscar_decode_step": (I32, [P, P, P, P, P, I32, I32, P, P, ctypes.c_size_t, P]),
            "oscar_decode_step_rope": (I32, [P, P, P, P, P, I32, I32, D, P, P, ctypes.c_size_t, P]),
            "oscar_decode_step_host_staging_size": (ctypes.c_size_t, [P, I32]),
            "oscar_decode_step_host": (I32, [P, P, P, I32, I32, D, P, P, ctypes.c_size_t, P,
                                             ctypes.c_size_t, P]),
            "oscar_multiquery_attention": (I32, [P, P, P, P, I32, I32, I32, P, P, ctypes.c_size_t, P]),
            "oscar_calibration_workspace_size": (ctypes.c_size_t, [I32, I32, I32, I64]),
            "oscar_query_covariance_device": (I32, [I32, I32, I32, I64, P, P, P, ctypes.c_size_t, P]),
            "oscar_score_covariance_device": (I32, [I32, I32, I32, I64, P, P, P, P, P,
                                                    ctypes.c_size_t, P]),
            "oscar_clip_threshold_device": (I32, [I32, I32, I64, P, P, D, P, P, ctypes.c_size_t, P]),
            "oscar_kv8_place": (I32, [P, P, P, I64, I64, P, P, I32, I64, I32, P]),
            "oscar_kv8_gather": (I32, [P, P, P, P, I32, I64, I32, P, P, P]),
            "oscar_kv8_workspace_size": (ctypes.c_size_t, [P, I32, I32, I32]),
            "oscar_kv8_attention": (I32, [P, P, P, P, I32, I32, I32, P, P, ctypes.c_size_t, P]),
            "oscar_kv4_place": (I32, [P, P, P, I64, I64, P, P, I32, I64, I32, P]),
            "oscar_kv4_gather": (I32, [P, P, P, P, I32, I64, I32, P, P, P]),
            "oscar_kv4_workspace_size": (ctypes.c_size_t, [P, I32, I32, I32]),
            "oscar_kv4_attention": (I32, [P, P, P, P, I32, I32, I32, P, P, ctypes.c_size_t, P]),
            "oscar_gather": (I32, [P, P, P, P, I32, I64, I32, P, P, P]),
            "oscar_extend_pages": (I32, [P, I32, P, P, I32, I32, P, I64, P, P, P, P, P, P, P, I64, P,
                                         P]),
            "oscar_rope_phases": (I32, [D, I32, D, I32, D, D, P]),
            "oscar_rope": (I32, [P, P, P, P, I64, I32, I32, I32, I32, I32, ctypes.c_float, I32, I64,
                                 I64, I64, I64, P, P, P]),
            "oscar_status_string": (ctypes.c_char_p, [I32]),
            "oscar_version": (I32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(fn: str, status: int) -> None:
    if status != OSCAR_OK:
        raise OscarError(fn, status)


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


# ------------------------------------------------------------------ host calls

def oscar_query_covariance(q: np.ndarray) -> np.ndarray:
    q = np.ascontiguousarray(q, np.float32)
    n, g, d = q.shape
    c = np.zeros((d, d), np.float64)
    _check("oscar_query_covariance", lib().oscar_query_covariance(d, g, n, _np_ptr(q), _np_ptr(c)))
    return c


def oscar_score_covariance(q: np.ndarray, k: np.ndarray, v: np.ndarray, num_threads: int = 0):
    q = np.ascontiguousarray(q, np.float32)
    k = np.ascontiguousarray(k, np.float32)
    v = np.ascontiguousarray(v, np.float32)
    n, g, d = q.shape
    c = np.zeros((d, d), np.float64)
    _check("oscar_score_covariance",
           lib().oscar_score_covariance(d, g, n, _np_ptr(q), _np_ptr(k), _np_ptr(v), num_threads,
                                        _np_ptr(c)))
    return c


def oscar_build_rotation(c, calib_x: np.ndarray, percentile: float = 99.9,
                         variant: int = VARIANT_OSCAR):
    """Returns (R64 [d,d] fp64, R32 [d,d] fp32, clip float32, eigenvalues [d])."""
    x = np.ascontiguousarray(calib_x, np.float32)
    n, d = x.shape
    cc = None if c is None else np.ascontiguousarray(c, np.float64)
    r64 = np.zeros((d, d), np.float64)
    r32 = np.zeros((d, d), np.float32)
    clip = np.zeros(1, np.float32)
    ev = np.zeros(d, np.float64)
    _check("oscar_build_rotation",
           lib().oscar_build_rotation(d, None if cc is None else _np_ptr(cc), _np_ptr(x), n,
                                      float(percentile), variant, _np_ptr(r64), _np_ptr(r32),
                                      _np_ptr(clip), _np_ptr(ev)))
    return r64, r32, np.float32(clip[0]), ev


# --------------------------------------------------------------- device calls

def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


@dataclasses.dataclass
class Cache:
    """Device tensors of one layer's cache plus its C descriptor.

    int2_pool: uint8 [num_int2_pages * Hkv * 12d] (INT4 variant, code_bits 4:
    20d per page-head); bf16_pool: bfloat16 [num_bf16_pages * Hkv * 32d]; page
    tables int32 [batch, max_pages_per_seq]; r_k, r_v fp32 [Hkv, d, d]; clip_k,
    clip_v fp32 [Hkv]; status int32 [1].
    """
    num_kv_heads: int
    num_q_heads: int
    head_dim: int
    sink: int
    window: int
    int2_pool: object
    bf16_pool: object
    int2_page_table: object
    bf16_page_table: object
    r_k: object = None
    r_v: object = None
    clip_k: object = None
    clip_v: object = None
    status: object = None
    code_bits: int = 2

    def desc(self) -> CacheDesc:
        # made again when a field, a tensor or the size of a pool or table has changed (each attribute
        # read once: 2.6 us on the host, as a loop over the tensors 4.6)
        codes, plain, table, plain_table = (self.int2_pool, self.bf16_pool, self.int2_page_table,
                                            self.bf16_page_table)
        rk, rv, ck, cv, status = self.r_k, self.r_v, self.clip_k, self.clip_v, self.status
        key = (None if codes is None else codes.data_ptr(), 0 if codes is None else codes.numel(),
               plain.data_ptr(), plain.numel(), None if table is None else table.data_ptr(),
               plain_table.data_ptr(), plain_table.shape, None if rk is None else rk.data_ptr(),
               None if rv is None else rv.data_ptr(), None if ck is None else ck.data_ptr(),
               None if cv is None else cv.data_ptr(), None if status is None else status.data_ptr(),
               self.num_kv_heads, self.num_q_heads, self.head_dim, self.sink, self.window,
               self.code_bits)
        cached = self.__dict__.get("_desc")
        if cached is not None and cached[0] == key:
            return cached[1]
        d = self.head_dim
        desc = CacheDesc(
            self.num_kv_heads, self.num_q_heads, d, self.sink, self.window,
            int(self.bf16_page_table.shape[1]),
            0 if self.int2_pool is None
            else self.int2_pool.numel() // (self.num_kv_heads * (4 * self.code_bits + 4) * d),
            self.bf16_pool.numel() // (self.num_kv_heads * 32 * d),
            _ptr(self.int2_pool), _ptr(self.bf16_pool), _ptr(self.int2_page_table),
            _ptr(self.bf16_page_table), _ptr(self.r_k), _ptr(self.r_v), _ptr(self.clip_k),
            _ptr(self.clip_v), _ptr(self.status), self.code_bits)
        self.__dict__["_desc"] = (key, desc)
        return desc


def oscar_prefill_quantize(cache: Cache, k, v, seq_ids, positions, seq_lens_final, stream=None):
    d = cache.desc()
    _check("oscar_prefill_quantize",
           lib().oscar_prefill_quantize(ctypes.byref(d), _ptr(k), _ptr(v), _ptr(seq_ids),
                                        _ptr(positions), _ptr(seq_lens_final),
                                        int(seq_lens_final.numel()), int(seq_ids.numel()),
                                        _stream(stream)))


def oscar_quantize_append(cache: Cache, k_new, v_new, seq_lens_after, stream=None):
    d = cache.desc()
    _check("oscar_quantize_append",
           lib().oscar_quantize_append(ctypes.byref(d), _ptr(k_new), _ptr(v_new),
                                       _ptr(seq_lens_after), int(seq_lens_after.numel()),
                                       _stream(stream)))


def oscar_prefill_quantize_trace(cache: Cache, k, v, seq_ids, positions, seq_lens_final, y_out,
                                 stream=None):
    """oscar_prefill_quantize that also writes the fp32 rotated values of every
    INT2 placement to y_out (float32 [total_tokens, Hkv, 2, d], device)."""
    d = cache.desc()
    _check("oscar_prefill_quantize_trace",
           lib().oscar_prefill_quantize_trace(ctypes.byref(d), _ptr(k), _ptr(v), _ptr(seq_ids),
                                              _ptr(positions), _ptr(seq_lens_final),
                                              int(seq_lens_final.numel()), int(seq_ids.numel()),
                                              _ptr(y_out), _stream(stream)))


def oscar_quantize_append_trace(cache: Cache, k_new, v_new, seq_lens_after, y_out, stream=None):
    """oscar_quantize_append that also writes the fp32 rotated values of each
    token leaving the window to y_out (float32 [batch, Hkv, 2, d], device)."""
    d = cache.desc()
    _check("oscar_quantize_append_trace",
           lib().oscar_quantize_append_trace(ctypes.byref(d), _ptr(k_new), _ptr(v_new),
                                             _ptr(seq_lens_after), int(seq_lens_after.numel()),
                                             _ptr(y_out), _stream(stream)))


def oscar_decode_workspace_size(cache: Cache, batch: int, max_seq_len: int) -> int:
    d = cache.desc()
    return int(lib().oscar_decode_workspace_size(ctypes.byref(d), batch, max_seq_len))


def oscar_multiquery_workspace_size(cache: Cache, batch: int, m_rows: int, max_seq_len: int) -> int:
    d = cache.desc()
    return int(lib().oscar_multiquery_workspace_size(ctypes.byref(d), batch, m_rows, max_seq_len))


def oscar_decode_attention(cache: Cache, q, seq_lens, max_seq_len: int, out, workspace,
                           stream=None):
    d = cache.desc()
    _check("oscar_decode_attention",
           lib().oscar_decode_attention(ctypes.byref(d), _ptr(q), _ptr(seq_lens),
                                        int(seq_lens.numel()), int(max_seq_len), _ptr(out),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)))


def oscar_decode_attention_bf16(cache: Cache, q, seq_lens, max_seq_len: int, out, workspace,
                                stream=None):
    d = cache.desc()
    _check("oscar_decode_attention_bf16",
           lib().oscar_decode_attention_bf16(ctypes.byref(d), _ptr(q), _ptr(seq_lens),
                                             int(seq_lens.numel()), int(max_seq_len), _ptr(out),
                                             _ptr(workspace),
                                             workspace.numel() * workspace.element_size(),
                                             _stream(stream)))


def oscar_decode_step(cache: Cache, q, k_new, v_new, seq_lens_after, max_seq_len: int, out,
                      workspace, stream=None):
    """Append the step's new token (and move the one leaving the window to INT2),
    then attend at the new lengths: one fused call, same result as
    oscar_quantize_append followed by oscar_decode_attention."""
    d = cache.desc()
    _check("oscar_decode_step",
           lib().oscar_decode_step(ctypes.byref(d), _ptr(q), _ptr(k_new), _ptr(v_new),
                                   _ptr(seq_lens_after), int(seq_lens_after.numel()),
                                   int(max_seq_len), _ptr(out), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)))


def oscar_decode_step_rope(cache: Cache, q, k_new, v_new, seq_lens_after, max_seq_len: int,
                           rope_base: float, out, workspace, stream=None):
    """The fused decode step with the rotary embedding of the new query and key."""
    d = cache.desc()
    _check("oscar_decode_step_rope",
           lib().oscar_decode_step_rope(ctypes.byref(d), _ptr(q), _ptr(k_new), _ptr(v_new),
                                        _ptr(seq_lens_after), int(seq_lens_after.numel()),
                                        int(max_seq_len), float(rope_base), _ptr(out),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)))


def oscar_decode_step_host_staging_size(cache: Cache, batch: int) -> int:
    """Device staging bytes of oscar_decode_step_host for `batch` sequences."""
    return int(lib().oscar_decode_step_host_staging_size(ctypes.byref(cache.desc()), int(batch)))


def oscar_decode_step_host(cache: Cache, in_host, seq_lens_after, max_seq_len: int, out_host,
                           staging, workspace, rope_base: float = 0.0, stream=None):
    """The fused decode step with its inputs and result in host memory.

    in_host: host bf16 tensor holding q [B][Hq][d], k_new [B][Hkv][d] and
    v_new [B][Hkv][d] back to back (pinned for asynchronous copies); out_host:
    host bf16 [B][Hq][d]; staging, workspace: device bytes.  Everything is
    queued on the stream; synchronise it before reading out_host."""
    d = cache.desc()
    _check("oscar_decode_step_host",
           lib().oscar_decode_step_host(ctypes.byref(d), _ptr(in_host), _ptr(seq_lens_after),
                                        int(seq_lens_after.numel()), int(max_seq_len),
                                        float(rope_base), _ptr(out_host), _ptr(staging),
                                        staging.numel() * staging.element_size(), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream)))


def oscar_multiquery_attention(cache: Cache, q, seq_lens, q_pos, max_seq_len: int, out, workspace,
                               stream=None):
    """Several query rows per sequence (q [B][M][Hq][d], q_pos [B][M]) over the
    mixed cache; row (b, m) attends to stored tokens 0 .. q_pos[b][m]."""
    d = cache.desc()
    B, M = int(q_pos.shape[0]), int(q_pos.shape[1])
    _check("oscar_multiquery_attention",
           lib().oscar_multiquery_attention(ctypes.byref(d), _ptr(q), _ptr(seq_lens), _ptr(q_pos),
                                            B, M, int(max_seq_len), _ptr(out), _ptr(workspace),
                                            workspace.numel() * workspace.element_size(),
                                            _stream(stream)))


def oscar_decode_attention_static(cache: Cache, q, seq_lens, max_seq_len: int, out, stream=None):
    """Decode attention without a workspace argument, for callers that cannot
    allocate device memory: the library's own fixed 16 MiB scratch buffer is
    used and nothing is allocated.  Calls must not overlap on the GPU."""
    d = cache.desc()
    _check("oscar_decode_attention_static",
           lib().oscar_decode_attention_static(ctypes.byref(d), _ptr(q), _ptr(seq_lens),
                                               int(seq_lens.numel()), int(max_seq_len), _ptr(out),
                                               _stream(stream)))


def oscar_calibration_workspace_size(num_kv_heads: int, num_q_heads: int, d: int, n: int) -> int:
    return int(lib().oscar_calibration_workspace_size(num_kv_heads, num_q_heads, d, n))


def _ws_bytes(workspace) -> int:
    return workspace.numel() * workspace.element_size()


def oscar_query_covariance_device(q, num_kv_heads: int, c_out, workspace, stream=None):
    """C_Q per KV head on the device: q bf16 [n][Hq][d] -> c_out fp64 [Hkv][d][d]."""
    n, hq, d = (int(x) for x in q.shape)
    _check("oscar_query_covariance_device",
           lib().oscar_query_covariance_device(num_kv_heads, hq, d, n, _ptr(q), _ptr(c_out),
                                               _ptr(workspace), _ws_bytes(workspace),
                                               _stream(stream)))


def oscar_score_covariance_device(q, k, v, c_out, workspace, stream=None):
    """C_S per KV head on the device: q bf16 [n][Hq][d], k/v bf16 [n][Hkv][d]."""
    n, hq, d = (int(x) for x in q.shape)
    hkv = int(k.shape[1])
    _check("oscar_score_covariance_device",
           lib().oscar_score_covariance_device(hkv, hq, d, n, _ptr(q), _ptr(k), _ptr(v),
                                               _ptr(c_out), _ptr(workspace), _ws_bytes(workspace),
                                               _stream(stream)))


def oscar_clip_threshold_device(x, r, percentile: float, clip_out, workspace, stream=None):
    """Clip per KV head on the device: x bf16 [n][Hkv][d], r fp32 [Hkv][d][d]."""
    n, hkv, d = (int(x_) for x_ in x.shape)
    _check("oscar_clip_threshold_device",
           lib().oscar_clip_threshold_device(hkv, d, n, _ptr(x), _ptr(r), float(percentile),
                                             _ptr(clip_out), _ptr(workspace), _ws_bytes(workspace),
                                             _stream(stream)))


# ---------------- 8-bit and 4-bit cache, reading back, page tables, rotary positions
#
# These calls check their tensors (type, shape, strides, one device) and raise
# ValueError; what the tensors hold is checked by the kernels.  They run on the
# device of their tensors, on `stream` or that device's current stream.

def _need(ok: bool, fn: str, what: str) -> None:
    if not ok:
        raise ValueError(f"{fn}: {what}")


# A decode step's calls take less time on the GPU than checks written at leisure take
# on the host: each of these reads an attribute of a tensor once, and a message is put
# together only when it is raised.

_INT32 = _INT64 = _BF16 = _FP32 = _raw_stream = _current_device = None


def _bind_torch() -> None:
    """What the checks use of torch, which is imported when the first tensor comes."""
    global _INT32, _INT64, _BF16, _FP32, _raw_stream, _current_device
    import torch
    _INT32, _INT64, _BF16, _FP32 = torch.int32, torch.int64, torch.bfloat16, torch.float32
    # the current stream's handle without a Stream object around it
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _i32(fn: str, name: str, t, index: int) -> int:
    """The address of a contiguous int32 tensor on CUDA device `index`."""
    if t.dtype is not _INT32 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous int32 tensor on cuda:{index}")
    return t.data_ptr()


def _rows(fn: str, name: str, t, n: int, heads: int, d: int, index: int) -> int:
    """Row stride in elements of a bf16 tensor [n][heads][d] whose rows are contiguous."""
    if t.dtype is not _BF16 or t.get_device() != index or t.shape != (n, heads, d):
        raise ValueError(f"{fn}: {name} must be a bfloat16 tensor [{n}][{heads}][{d}] on cuda:{index}")
    row, head, one = t.stride()
    if (one != 1 and d > 1) or (head != d and heads > 1):
        raise ValueError(f"{fn}: {name}: the heads of a row must be contiguous")
    return row if n > 1 else heads * d


def _fits(fn: str, name: str, value: int) -> int:
    """An argument that the library takes as int32: ctypes would cut it."""
    if not -0x80000000 <= value <= 0x7fffffff:
        raise ValueError(f"{fn}: {name} is outside the range of int32")
    return value


def _device_of(fn: str, name: str, t) -> int:
    if _INT32 is None:
        _bind_torch()
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{fn}: {name} must be on a CUDA device")
    return index


def _launch(fn: str, index: int, stream, *args) -> None:
    """Calls the library's `fn` with the stream appended, with device `index` current."""
    f = getattr(_LIB or lib(), fn)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        status = f(*args, handle)
    else:
        import torch
        with torch.cuda.device(index):
            status = f(*args, handle)
    if status != OSCAR_OK:
        raise OscarError(fn, status)


def oscar_gather(cache: Cache, seq_lens, first, row_starts, max_rows: int, k_out, v_out, stream=None):
    """Read tokens of the calibrated cache back as bf16: rows row_starts[b] .. row_starts[b+1] - 1
    of k_out and v_out (contiguous [n][Hkv][d]) get sequence b's tokens from position first[b] on,
    BF16 ones as stored, INT2 or INT4 ones as code * s + z, rotated back."""
    fn = "oscar_gather"
    if cache.int2_pool is None or cache.bf16_pool is None:
        raise ValueError(f"{fn}: the cache must have both pools")
    index = _device_of(fn, "int2_pool", cache.int2_pool)
    d = cache.desc()
    n, h, dim = k_out.shape[0], cache.num_kv_heads, cache.head_dim
    if (_rows(fn, "k_out", k_out, n, h, dim, index) != h * dim
            or _rows(fn, "v_out", v_out, n, h, dim, index) != h * dim):
        raise ValueError(f"{fn}: k_out and v_out must be contiguous")
    lens, begin = _i32(fn, "seq_lens", seq_lens, index), _i32(fn, "first", first, index)
    starts = _i32(fn, "row_starts", row_starts, index)
    coded, plain = cache.int2_page_table, cache.bf16_page_table
    _i32(fn, "int2_page_table", coded, index)
    _i32(fn, "bf16_page_table", plain, index)
    if cache.status is not None:
        _i32(fn, "status", cache.status, index)
    batch, shape = seq_lens.numel(), coded.shape
    if first.numel() != batch or row_starts.numel() != batch + 1:
        raise ValueError(f"{fn}: first must have batch entries, row_starts batch + 1")
    if shape != plain.shape or len(shape) != 2 or batch > shape[0]:
        raise ValueError(f"{fn}: the page tables must have the same shape, and a row per sequence")
    for pool, size in ((cache.int2_pool, 1), (cache.bf16_pool, 2)):
        if pool.get_device() != index or pool.element_size() != size or not pool.is_contiguous():
            raise ValueError(f"{fn}: int2_pool and bf16_pool must be contiguous tensors of bytes and of "
                             f"bfloat16 on cuda:{index}")
    for r in (cache.r_k, cache.r_v):
        if (r is None or r.get_device() != index or r.dtype is not _FP32 or r.numel() != h * dim * dim
                or not r.is_contiguous()):
            raise ValueError(f"{fn}: r_k and r_v must be contiguous float32 tensors [{h}][{dim}][{dim}] "
                             f"on cuda:{index}")
    _launch(fn, index, stream, ctypes.byref(d), lens, begin, starts, batch, n,
            _fits(fn, "max_rows", max_rows), k_out.data_ptr(), v_out.data_ptr())


class _PagedCache:
    """What the 8-bit and the 4-bit cache share: checked tensors and a C descriptor."""
    fmt = None   # Kv8Cache: which 8 bits

    def desc(self):
        return self._checked()[0]

    def _checked(self):
        """(descriptor, a pointer to it, device index, page-table rows), checked again when a
        tensor or a field has been replaced."""
        pool, tail, table, ids, status = (self.pool, self.tail, self.page_table, self.tail_ids,
                                          self.status)
        key = (pool.data_ptr(), pool.shape, pool.dtype, pool.is_contiguous(),
               tail.data_ptr(), tail.shape, tail.dtype, tail.is_contiguous(),
               table.data_ptr(), table.shape, table.dtype, table.is_contiguous(),
               None if ids is None else (ids.data_ptr(), ids.shape, ids.dtype, ids.is_contiguous()),
               None if status is None else (status.data_ptr(), status.dtype),
               self.fmt, self.num_q_heads, self.num_kv_heads, self.head_dim)
        cached = self.__dict__.get("_desc")
        if cached is not None and cached[0] == key:
            return cached[1]
        import torch
        fn, h, d = type(self).__name__, self.num_kv_heads, self.head_dim
        size = self._block_bytes(d)
        index = _device_of(fn, "pool", self.pool)
        _need(self.pool.dtype is torch.uint8 and self.pool.is_contiguous()
              and self.pool.shape[1:] == (h, size), fn,
              f"pool must be a contiguous uint8 tensor [num_pages][{h}][{size}]")
        _need(self.tail.dtype is torch.bfloat16 and self.tail.is_contiguous()
              and self.tail.get_device() == index and self.tail.shape[1:] == (h, 2, 16 * d), fn,
              f"tail must be a contiguous bfloat16 tensor [num_tails][{h}][2][{16 * d}] on cuda:{index}")
        _i32(fn, "page_table", self.page_table, index)
        _need(self.page_table.dim() == 2, fn, "page_table must be [batch][max_pages_per_seq]")
        rows = int(self.page_table.shape[0])
        if self.tail_ids is not None:
            _i32(fn, "tail_ids", self.tail_ids, index)
            _need(self.tail_ids.numel() == rows, fn,
                  "tail_ids must have an entry per row of the page table")
        if self.status is not None:
            _i32(fn, "status", self.status, index)
        desc = self._make_desc(h, self.num_q_heads, d, int(self.page_table.shape[1]),
                               int(self.pool.shape[0]), int(self.tail.shape[0]), _ptr(self.pool),
                               _ptr(self.tail), _ptr(self.page_table), _ptr(self.tail_ids),
                               _ptr(self.status))
        found = (desc, ctypes.byref(desc), index, rows)
        self.__dict__["_desc"] = (key, found)
        return found


@dataclasses.dataclass
class Kv8Cache(_PagedCache):
    """Device tensors of one layer's 8-bit cache plus its C descriptor.

    pool: uint8 [num_pages, Hkv, 32d + 16]; tail: bfloat16 [num_tails, Hkv, 2, 16d];
    page_table: int32 [batch, max_pages_per_seq]; tail_ids: int32 [batch] or None
    (sequence b has tail block b); status: int32 [1] or None; fmt: KV8_INT8 or
    KV8_E4M3.  ``pages.allocate_kv8`` makes one.
    """
    num_kv_heads: int
    num_q_heads: int
    head_dim: int
    pool: object
    tail: object
    page_table: object
    fmt: int = KV8_INT8
    tail_ids: object = None
    status: object = None

    @staticmethod
    def _block_bytes(d: int) -> int:
        return 32 * d + 16

    def _make_desc(self, *fields) -> Kv8Desc:
        return Kv8Desc(*fields, self.fmt)


@dataclasses.dataclass
class Kv4Cache(_PagedCache):
    """Device tensors of one layer's 4-bit cache plus its C descriptor.

    pool: uint8 [num_pages, Hkv, 18d + 16]; the others as ``Kv8Cache``'s.
    ``pages.allocate_kv4`` makes one.
    """
    num_kv_heads: int
    num_q_heads: int
    head_dim: int
    pool: object
    tail: object
    page_table: object
    tail_ids: object = None
    status: object = None

    @staticmethod
    def _block_bytes(d: int) -> int:
        return 18 * d + 16

    @staticmethod
    def _make_desc(*fields) -> Kv4Desc:
        return Kv4Desc(*fields)


def _checked_cache(fn: str, cache, kind):
    if not isinstance(cache, kind):
        raise ValueError(f"{fn}: cache must be a {kind.__name__}")
    return cache._checked()


def _place(fn, kind, cache, k, v, lens_before, row_starts, max_new, stream):
    _, desc, index, rows = _checked_cache(fn, cache, kind)
    n, h, d = k.shape[0], cache.num_kv_heads, cache.head_dim
    ks = _rows(fn, "k", k, n, h, d, index)
    vs = _rows(fn, "v", v, n, h, d, index)
    lens, starts = _i32(fn, "lens_before", lens_before, index), _i32(fn, "row_starts", row_starts, index)
    batch = lens_before.numel()
    if row_starts.numel() != batch + 1 or batch > rows:
        raise ValueError(f"{fn}: row_starts must have batch + 1 entries, and the page table a row "
                         "per sequence")
    _launch(fn, index, stream, desc, k.data_ptr(), v.data_ptr(), ks, vs, lens, starts, batch, n,
            _fits(fn, "max_new", max_new))


def _gather(fn, kind, cache, seq_lens, first, row_starts, max_rows, k_out, v_out, stream):
    _, desc, index, rows = _checked_cache(fn, cache, kind)
    n, h, d = k_out.shape[0], cache.num_kv_heads, cache.head_dim
    if (_rows(fn, "k_out", k_out, n, h, d, index) != h * d
            or _rows(fn, "v_out", v_out, n, h, d, index) != h * d):
        raise ValueError(f"{fn}: k_out and v_out must be contiguous")
    lens, begin = _i32(fn, "seq_lens", seq_lens, index), _i32(fn, "first", first, index)
    starts = _i32(fn, "row_starts", row_starts, index)
    batch = seq_lens.numel()
    if first.numel() != batch or row_starts.numel() != batch + 1 or batch > rows:
        raise ValueError(f"{fn}: first must have batch entries, row_starts batch + 1, and the page "
                         "table a row per sequence")
    _launch(fn, index, stream, desc, lens, begin, starts, batch, n, _fits(fn, "max_rows", max_rows),
            k_out.data_ptr(), v_out.data_ptr())


def _workspace_size(fn, kind, cache, batch, m_rows, max_seq_len) -> int:
    import torch
    _, desc, index, _ = _checked_cache(fn, cache, kind)
    for name, value in (("batch", batch), ("m_rows", m_rows), ("max_seq_len", max_seq_len)):
        _fits(fn, name, value)
    with torch.cuda.device(index):   # its number of SMs counts
        return int(getattr(lib(), fn)(desc, batch, m_rows, max_seq_len))


def _attention(fn, kind, cache, q, seq_lens, max_seq_len, out, workspace, q_pos, stream):
    _, desc, index, rows = _checked_cache(fn, cache, kind)
    lens, batch = _i32(fn, "seq_lens", seq_lens, index), seq_lens.numel()
    if q_pos is None:
        m_rows, pos, shape = 1, None, (batch, cache.num_q_heads, cache.head_dim)
    else:
        pos = _i32(fn, "q_pos", q_pos, index)
        if q_pos.dim() != 2 or q_pos.shape[0] != batch:
            raise ValueError(f"{fn}: q_pos must be [batch][rows]")
        m_rows = q_pos.shape[1]
        shape = (batch, m_rows, cache.num_q_heads, cache.head_dim)
    for t in (q, out):
        if (t.dtype is not _BF16 or t.get_device() != index or t.shape != shape
                or not t.is_contiguous()):
            raise ValueError(f"{fn}: q and out must be contiguous bfloat16 tensors {list(shape)} "
                             f"on cuda:{index}")
    if batch > rows or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"{fn}: the page table must have a row per sequence, and the workspace be "
                         f"a contiguous tensor on cuda:{index}")
    _launch(fn, index, stream, desc, q.data_ptr(), lens, pos, batch, m_rows,
            _fits(fn, "max_seq_len", max_seq_len),
            out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())


def oscar_kv8_place(cache: Kv8Cache, k, v, lens_before, row_starts, max_new: int, stream=None):
    """Place the rows of k and v (bf16 [n][Hkv][d], rows may be strided): sequence b's
    rows row_starts[b] .. row_starts[b+1] - 1 go behind its lens_before[b] tokens.
    max_new: the most rows that one sequence brings."""
    _place("oscar_kv8_place", Kv8Cache, cache, k, v, lens_before, row_starts, max_new, stream)


def oscar_kv8_gather(cache: Kv8Cache, seq_lens, first, row_starts, max_rows: int, k_out, v_out,
                     stream=None):
    """Read tokens back as bf16: rows row_starts[b] .. row_starts[b+1] - 1 of k_out and
    v_out (contiguous [n][Hkv][d]) get sequence b's tokens from position first[b] on."""
    _gather("oscar_kv8_gather", Kv8Cache, cache, seq_lens, first, row_starts, max_rows, k_out, v_out,
            stream)


def oscar_kv8_workspace_size(cache: Kv8Cache, batch: int, m_rows: int, max_seq_len: int) -> int:
    """Bytes for oscar_kv8_attention of no more sequences, rows and tokens; 0: invalid."""
    return _workspace_size("oscar_kv8_workspace_size", Kv8Cache, cache, batch, m_rows, max_seq_len)


def oscar_kv8_attention(cache: Kv8Cache, q, seq_lens, max_seq_len: int, out, workspace, q_pos=None,
                        stream=None):
    """Attention over the 8-bit cache.  Decode: q, out bf16 [B][Hq][d], every row sees
    the seq_lens[b] tokens stored.  With q_pos (int32 [B][M]): q, out [B][M][Hq][d],
    row (b, m) sees positions 0 .. q_pos[b][m] (negative: a padded row, zeros).
    max_seq_len decides the form of the kernel: announce no more than is needed."""
    _attention("oscar_kv8_attention", Kv8Cache, cache, q, seq_lens, max_seq_len, out, workspace, q_pos,
               stream)


def oscar_kv4_place(cache: Kv4Cache, k, v, lens_before, row_starts, max_new: int, stream=None):
    """oscar_kv8_place into a 4-bit cache."""
    _place("oscar_kv4_place", Kv4Cache, cache, k, v, lens_before, row_starts, max_new, stream)


def oscar_kv4_gather(cache: Kv4Cache, seq_lens, first, row_starts, max_rows: int, k_out, v_out,
                     stream=None):
    """oscar_kv8_gather from a 4-bit cache."""
    _gather("oscar_kv4_gather", Kv4Cache, cache, seq_lens, first, row_starts, max_rows, k_out, v_out,
            stream)


def oscar_kv4_workspace_size(cache: Kv4Cache, batch: int, m_rows: int, max_seq_len: int) -> int:
    """Bytes for oscar_kv4_attention of no more sequences, rows and tokens; 0: invalid."""
    return _workspace_size("oscar_kv4_workspace_size", Kv4Cache, cache, batch, m_rows, max_seq_len)


def oscar_kv4_attention(cache: Kv4Cache, q, seq_lens, max_seq_len: int, out, workspace, q_pos=None,
                        stream=None):
    """oscar_kv8_attention over a 4-bit cache."""
    _attention("oscar_kv4_attention", Kv4Cache, cache, q, seq_lens, max_seq_len, out, workspace, q_pos,
               stream)


def oscar_extend_pages(page_table, lens, new_tokens, free_pages, cursor, lens_after, page_starts,
                       row_starts, seq_ids, positions, slots=None, hold_back: int = 0, status=None,
                       stream=None):
    """Grow every sequence by new_tokens[b]: new page-table entries from free_pages
    (from index cursor[0] on), lengths, prefix sums and the lists of the new tokens.
    page_starts[B] is the next call's cursor (pass page_starts[-1:]); lens_after may
    be lens.  Rows of seq_ids, positions and slots behind the new tokens become -1."""
    fn = "oscar_extend_pages"
    index = _device_of(fn, "page_table", page_table)
    batch, rows = lens.numel(), seq_ids.numel()
    table, before = _i32(fn, "page_table", page_table, index), _i32(fn, "lens", lens, index)
    new, free = _i32(fn, "new_tokens", new_tokens, index), _i32(fn, "free_pages", free_pages, index)
    at, after = _i32(fn, "cursor", cursor, index), _i32(fn, "lens_after", lens_after, index)
    ps, rs = _i32(fn, "page_starts", page_starts, index), _i32(fn, "row_starts", row_starts, index)
    ids, pos = _i32(fn, "seq_ids", seq_ids, index), _i32(fn, "positions", positions, index)
    if page_table.dim() != 2 or page_table.shape[0] < batch:
        raise ValueError(f"{fn}: page_table must be [batch][max_pages_per_seq]")
    if (new_tokens.numel() != batch or lens_after.numel() != batch or cursor.numel() < 1
            or page_starts.numel() != batch + 1 or row_starts.numel() != batch + 1):
        raise ValueError(f"{fn}: new_tokens and lens_after must have batch entries, page_starts and "
                         "row_starts batch + 1, cursor one")
    if positions.numel() != rows:
        raise ValueError(f"{fn}: seq_ids and positions must have the same rows")
    if slots is not None and (slots.dtype is not _INT64 or slots.get_device() != index
                              or not slots.is_contiguous() or slots.numel() != rows):
        raise ValueError(f"{fn}: slots must be a contiguous int64 tensor on cuda:{index} with a "
                         "row per seq_ids row")
    _launch(fn, index, stream, table, page_table.shape[1], before, new, batch,
            _fits(fn, "hold_back", hold_back), free,
            free_pages.numel(), at, after, ps, rs, ids, pos, _ptr(slots), rows,
            None if status is None else _i32(fn, "status", status, index))


def oscar_rope_phases(base: float, rotary_dim: int, factor: float = 1.0, original_len: int = 0,
                      low_turns: float = 1.0, high_turns: float = 32.0) -> np.ndarray:
    """Rotary frequencies of oscar_rope, uint64 [rotary_dim / 2] (turns per token times
    2^64): unscaled, divided by `factor`, or (original_len > 0) scaled by parts, with a
    ramp that is linear in the turns over original_len (not in the pair's index, as
    some models have it: their words are the caller's to form)."""
    for name, value in (("rotary_dim", rotary_dim), ("original_len", original_len)):
        _fits("oscar_rope_phases", name, int(value))
    out = np.zeros(max(int(rotary_dim) // 2, 1), np.uint64)
    _check("oscar_rope_phases",
           lib().oscar_rope_phases(float(base), int(rotary_dim), float(factor), int(original_len),
                                   float(low_turns), float(high_turns), _np_ptr(out)))
    return out


def oscar_rope(q, k, positions, phases, q_out=None, k_out=None, interleaved: bool = False,
               amplitude: float = 1.0, inverse: bool = False, stream=None):
    """Rotary embedding of q [n][Hq][d] and k [n][Hkv][d] (bf16, rows may be strided;
    either may be None) at int32 positions [n] (negative: the row is left as it was).
    phases: oscar_rope_phases' words on the device as int64 (or uint64) [rotary_dim / 2].
    q_out, k_out: outputs, in place when None."""
    fn = "oscar_rope"
    some = k if q is None else q
    if some is None or some.dim() != 3:
        raise ValueError(f"{fn}: q or k must be given, as [n][heads][d]")
    index = _device_of(fn, "q and k", some)
    n, _, d = some.shape
    hq = hk = qs = ks = qos = kos = 0
    qp = kp = qop = kop = None
    if q is not None:
        hq = q.shape[1]
        qs = qos = _rows(fn, "q", q, n, hq, d, index)
        qp = qop = q.data_ptr()
        if q_out is not None:
            qos, qop = _rows(fn, "q_out", q_out, n, hq, d, index), q_out.data_ptr()
    if k is not None:
        hk = k.shape[1]
        ks = kos = _rows(fn, "k", k, n, hk, d, index)
        kp = kop = k.data_ptr()
        if k_out is not None:
            kos, kop = _rows(fn, "k_out", k_out, n, hk, d, index), k_out.data_ptr()
    pos = _i32(fn, "positions", positions, index)
    if positions.numel() != n or (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError(f"{fn}: positions must have an entry per row, and an output its input")
    if ((phases.dtype is not _INT64 and str(phases.dtype) != "torch.uint64")
            or phases.get_device() != index or not phases.is_contiguous()):
        raise ValueError(f"{fn}: phases must be contiguous 64-bit integers on cuda:{index}")
    _launch(fn, index, stream, qp, kp, pos, phases.data_ptr(), n, hq, hk, d, 2 * phases.numel(),
            1 if interleaved else 0, amplitude, 1 if inverse else 0, qs, ks, qos, kos, qop, kop)


def oscar_device_sm_count() -> int:
    return int(lib().oscar_device_sm_count())


def oscar_version() -> int:
    return int(lib().oscar_version())

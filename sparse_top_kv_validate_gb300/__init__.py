"""GB300 KV-cache attention library: Python binding of ``libsa.so``.

This module only marshals arguments: it turns torch CUDA tensors into the
device pointers and sizes of the C ABI declared in ``include/sa.h`` and
passes torch's current stream.  Every step of the computation runs in the
library's CUDA kernels; if ``libsa.so`` is missing the calls raise instead of
falling back to anything else.

Entry points (same names as the C ABI):
    validate_indices, build_present_kv, sparse_attn_decode, attn_prefill,
    paged_attn_decode, sparse_index_select, csa_ratio4_attention,
    csa_ratio128_compress, csa_ratio4_main_compress, csa_ratio4_index_compress,
    csa_pool_weight, rotary_embed, paged_kv_write, paged_kv_read, attn_prefill_packed,
    attn_weights_packed, paged_attn_decode_weights (paged_attn_decode with weights),
    paged_kv_select, paged_kv_compact
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
import struct
import threading

import torch

__all__ = [
    "load", "lib_path", "SAError", "status_string", "check_wait_timeout", "graph_kernel_count",
    "validate_indices", "build_present_kv", "sparse_attn_decode", "attn_prefill",
    "paged_attn_decode", "sparse_attn_decode_workspace", "attn_prefill_workspace",
    "paged_attn_decode_workspace", "new_workspace", "sparse_attn_decode_noalloc",
    "NOALLOC_SCRATCH_BYTES", "ERR_SCRATCH_LIMIT", "OPT_ROW_COPIES", "OPT_FP8_WARP_MMA",
    "F32", "F16", "BF16", "FP8_E4M3_B64",
    "IDX_BELOW_SENTINEL", "IDX_AFTER_PADDING", "IDX_OUT_OF_RANGE", "IDX_NOT_INCREASING",
    "IDX_DUPLICATE", "IDX_ALL_PADDING", "ERRBIT_WRITE_POS", "ERRBIT_PAGE", "ERRBIT_TIMEOUT",
    "SparseParams", "PrefillParams", "PagedParams", "kernel_events",
    "IndexSelectParams", "sparse_index_select", "sparse_index_select_workspace",
    "SEL_TIE", "SEL_NONFINITE", "ERRBIT_SEL_TIE", "ERRBIT_SEL_NONFINITE",
    "CsaParams", "csa_ratio4_attention", "csa_ratio4_attention_workspace", "ERRBIT_RECORD",
    "CompressParams", "csa_ratio128_compress", "csa_ratio4_main_compress",
    "csa_ratio4_index_compress", "csa_pool_weight", "ERRBIT_COMPRESS",
    "RopeTable", "rope_table", "RotaryParams", "rotary_embed", "KvPagesParams", "paged_kv_write",
    "paged_kv_read", "new_fp8_pool", "PackedParams", "attn_prefill_packed", "FP8_E4M3_PAGE",
    "ERRBIT_SEQ", "ERRBIT_NONFINITE",
    "WeightsParams", "attn_weights_packed", "new_weight_pool", "SelectParams", "paged_kv_select",
    "CompactParams", "paged_kv_compact", "paged_attn_decode_weights_workspace",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = os.path.join(_HERE, "_build", "libsa.so")

F32, F16, BF16, FP8_E4M3_B64 = 0, 1, 2, 3
IDX_BELOW_SENTINEL, IDX_AFTER_PADDING, IDX_OUT_OF_RANGE = 1, 2, 4
IDX_NOT_INCREASING, IDX_DUPLICATE, IDX_ALL_PADDING = 8, 16, 32
ERRBIT_WRITE_POS, ERRBIT_PAGE, ERRBIT_TIMEOUT = 64, 128, 256
ERR_SCRATCH_LIMIT = -9
ERR_WORKSPACE = -5
NOALLOC_SCRATCH_BYTES = 16 << 20
OPT_ROW_COPIES, OPT_FP8_WARP_MMA = 1, 2
SEL_TIE, SEL_NONFINITE = 1, 2
ERRBIT_SEL_TIE, ERRBIT_SEL_NONFINITE = 512, 1024
ERRBIT_RECORD = 2048
ERRBIT_COMPRESS = 4096
FP8_E4M3_PAGE = 4
ERRBIT_SEQ, ERRBIT_NONFINITE = 8192, 16384

_p = C.c_void_p
_i64 = C.c_int64
_i32 = C.c_int32


class SparseParams(C.Structure):
    _fields_ = [
        ("q", _p), ("k_cache", _p), ("v_cache", _p), ("idx", _p), ("sink", _p), ("y", _p),
        ("q_dtype", _i32), ("kv_dtype", _i32), ("idx_is_i64", _i32), ("causal", _i32),
        ("B", _i64), ("Hq", _i64), ("Hkv", _i64), ("Sq", _i64), ("D", _i64), ("Dv", _i64),
        ("T", _i64), ("I", _i64), ("K", _i64),
        ("kv_len", _p), ("past_len", _i64),
        ("scale", C.c_float), ("softcap", C.c_float),
        ("window", _i64), ("record_stride", _i64), ("n_rope", _i64),
        ("err_word", _p), ("row_status", _p),
        ("k_cur", _p), ("v_cur", _p), ("write_pos", _p), ("cur_len", _i64),
        ("workspace", _p), ("workspace_bytes", C.c_size_t),
        ("bias", _p), ("bias_rank", _i64), ("bias_dims", _i64 * 4),
        ("options", C.c_uint32), ("reserved_", C.c_uint32),
    ]


class PrefillParams(C.Structure):
    _fields_ = [
        ("q", _p), ("k", _p), ("v", _p), ("y", _p), ("present_k", _p), ("present_v", _p),
        ("dtype", _i32), ("causal", _i32),
        ("B", _i64), ("Hq", _i64), ("Hkv", _i64), ("S", _i64), ("D", _i64),
        ("scale", C.c_float), ("softcap", C.c_float),
        ("workspace", _p), ("workspace_bytes", C.c_size_t), ("err_word", _p),
        ("attn_mask", _p), ("mask_kind", _i32), ("reserved_", _i32), ("mask_rank", _i64),
        ("mask_dims", _i64 * 4), ("nonpad_kv_seqlen", _p),
    ]


class PagedParams(C.Structure):
    _fields_ = [
        ("q", _p), ("k_pool", _p), ("v_pool", _p), ("k_new", _p), ("v_new", _p),
        ("block_table", _p), ("ctx_len", _p), ("y", _p),
        ("dtype", _i32), ("options", C.c_uint32),
        ("B", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64), ("page_tokens", _i64),
        ("max_pages", _i64), ("num_pages", _i64),
        ("scale", C.c_float), ("pool_format", _i32),
        ("err_word", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t),
    ]


class IndexSelectParams(C.Structure):
    _fields_ = [
        ("query", _p), ("weight", _p), ("keys", _p), ("selected", _p), ("row_status", _p),
        ("err_word", _p),
        ("B", _i64), ("S", _i64), ("IH", _i64), ("ID", _i64), ("R", _i64), ("topk", _i64),
        ("key_stride", _i64), ("out_heads", _i64), ("query_start", _i64),
        ("query_start_b", _p), ("ascending", _i32), ("reserved_", _i32),
        ("workspace", _p), ("workspace_bytes", C.c_size_t),
    ]


class CsaParams(C.Structure):
    _fields_ = [
        ("query", _p), ("current_kv", _p), ("records", _p), ("selected", _p), ("sink", _p),
        ("bias", _p), ("bias_rank", _i64), ("bias_dims", _i64 * 4), ("y", _p),
        ("q_dtype", _i32), ("kv_dtype", _i32),
        ("B", _i64), ("S", _i64), ("H", _i64), ("D", _i64), ("n_rope", _i64), ("L", _i64),
        ("R", _i64), ("topk", _i64), ("record_stride", _i64), ("total", _i64),
        ("scale", C.c_float), ("reserved_", _i32), ("err_word", _p),
        ("workspace", _p), ("workspace_bytes", C.c_size_t),
    ]


class CompressParams(C.Structure):
    _fields_ = [
        ("kv", _p), ("gate", _p), ("ape", _p), ("norm", _p), ("carry", _p), ("records", _p),
        ("logical", _p), ("err_word", _p),
        ("B", _i64), ("S", _i64), ("D", _i64), ("n_rope", _i64), ("rows", _i64),
        ("record_stride", _i64), ("total", _i64), ("reserved_", _i64),
    ]


class RopeTable(C.Structure):
    """Angles of the rotary pairs (``sa_rope``), made by ``rope_table``."""
    _fields_ = [("rotary_dim", _i32), ("interleaved", _i32), ("mscale", C.c_float),
                ("reserved_", _i32), ("turns", C.c_uint64 * 128)]


class _RopeConfig(C.Structure):
    _fields_ = [("rotary_dim", _i32), ("interleaved", _i32), ("scaling", _i32),
                ("mscale", C.c_float), ("base", C.c_double), ("factor", C.c_double),
                ("original_len", C.c_double), ("ramp_low", C.c_double),
                ("ramp_high", C.c_double), ("inv_freq", _p)]


class RotaryParams(C.Structure):
    _fields_ = [
        ("q", _p), ("k", _p), ("q_out", _p), ("k_out", _p), ("positions", _p), ("rope", _p),
        ("dtype", _i32), ("pos_is_i64", _i32),
        ("B", _i64), ("S", _i64), ("Hq", _i64), ("Hk", _i64), ("D", _i64), ("pos_stride", _i64),
        ("q_strides", _i64 * 3), ("k_strides", _i64 * 3), ("q_out_strides", _i64 * 3),
        ("k_out_strides", _i64 * 3),
    ]


class KvPagesParams(C.Structure):
    _fields_ = [
        ("k", _p), ("v", _p), ("k_pool", _p), ("v_pool", _p), ("block_table", _p),
        ("ctx_len", _p), ("seq_start", _p), ("rope", _p), ("err_word", _p),
        ("dtype", _i32), ("pool_format", _i32),
        ("T", _i64), ("B", _i64), ("Hkv", _i64), ("D", _i64), ("page_tokens", _i64),
        ("max_pages", _i64), ("num_pages", _i64), ("k_strides", _i64 * 2),
        ("v_strides", _i64 * 2),
    ]


class PackedParams(C.Structure):
    _fields_ = [
        ("q", _p), ("k", _p), ("v", _p), ("y", _p), ("q_start", _p), ("k_start", _p),
        ("err_word", _p), ("dtype", _i32), ("causal", _i32),
        ("B", _i64), ("Tq", _i64), ("Tk", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64),
        ("q_strides", _i64 * 2), ("k_strides", _i64 * 2), ("v_strides", _i64 * 2),
        ("y_strides", _i64 * 2), ("scale", C.c_float), ("softcap", C.c_float),
    ]


class WeightsParams(C.Structure):
    _fields_ = [
        ("q", _p), ("k", _p), ("weights", _p), ("block_table", _p), ("q_start", _p),
        ("k_start", _p), ("err_word", _p), ("dtype", _i32), ("accumulate", _i32),
        ("B", _i64), ("Tq", _i64), ("Tk", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64),
        ("page_tokens", _i64), ("max_pages", _i64), ("num_pages", _i64),
        ("q_strides", _i64 * 2), ("k_strides", _i64 * 2), ("scale", C.c_float),
        ("reserved_", _i32), ("workspace", _p), ("workspace_bytes", C.c_size_t),
    ]


class SelectParams(C.Structure):
    _fields_ = [
        ("weights", _p), ("block_table", _p), ("ctx_len", _p), ("keep", _p), ("new_len", _p),
        ("err_word", _p), ("B", _i64), ("Hkv", _i64), ("page_tokens", _i64), ("max_pages", _i64),
        ("num_pages", _i64), ("budget", _i64), ("sink", _i64), ("recent", _i64),
    ]


class CompactParams(C.Structure):
    _fields_ = [
        ("k_pool", _p), ("v_pool", _p), ("weights", _p), ("block_table", _p), ("ctx_len", _p),
        ("keep", _p), ("err_word", _p), ("dtype", _i32), ("pool_format", _i32),
        ("B", _i64), ("Hkv", _i64), ("D", _i64), ("page_tokens", _i64), ("max_pages", _i64),
        ("num_pages", _i64), ("width", _i64),
    ]


# The serving-step calls pack their parameters as bytes of the structures above (filling
# a ctypes structure field by field takes as long as the launch).
_ROTARY = struct.Struct("6P2i18q")
_KV_PAGES = struct.Struct("9P2i11q")
_PACKED = struct.Struct("7P2i14q2f")
_PAGED = struct.Struct("8PiI7qfi2PN")
_WEIGHTS = struct.Struct("7P2i13qfiPN")
_SELECT = struct.Struct("6P8q")
_COMPACT = struct.Struct("7P2i7q")


class SAError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call}: status {status} ({status_string(status)})")
        self.status = status


_lock = threading.Lock()
_lib = None


def lib_path() -> str:
    return _LIB


def load():
    """Load ``libsa.so`` (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB):
            raise RuntimeError(
                f"{_LIB} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        L = C.CDLL(_LIB)
        L.sa_status_string.restype = C.c_char_p
        L.sa_status_string.argtypes = [C.c_int]
        L.sa_version.restype = C.c_int
        L.sa_version.argtypes = []
        L.sa_set_kernel_events.restype = C.c_int
        L.sa_set_kernel_events.argtypes = [_p, _p]
        L.validate_indices.restype = C.c_int
        L.validate_indices.argtypes = [_p, C.c_int, _i64, _i64, _i64, _i64, _p, _i64, _p, _p, _p]
        L.build_present_kv.restype = C.c_int
        L.build_present_kv.argtypes = [_p, _p, _p, _p, _p, _p, C.c_int, _i64, _i64, _i64, _i64,
                                       _i64, _i64, _p, _p, _p]
        L.sparse_attn_decode_workspace.restype = C.c_size_t
        L.sparse_attn_decode_workspace.argtypes = [C.POINTER(SparseParams)]
        L.sparse_attn_decode.restype = C.c_int
        L.sparse_attn_decode.argtypes = [C.POINTER(SparseParams), _p]
        L.sparse_attn_decode_noalloc.restype = C.c_int
        L.sparse_attn_decode_noalloc.argtypes = [C.POINTER(SparseParams), _p]
        L.attn_prefill_workspace.restype = C.c_size_t
        L.attn_prefill_workspace.argtypes = [C.POINTER(PrefillParams)]
        L.attn_prefill.restype = C.c_int
        L.attn_prefill.argtypes = [C.POINTER(PrefillParams), _p]
        L.sparse_index_select_workspace.restype = C.c_size_t
        L.sparse_index_select_workspace.argtypes = [C.POINTER(IndexSelectParams)]
        L.sparse_index_select.restype = C.c_int
        L.sparse_index_select.argtypes = [C.POINTER(IndexSelectParams), _p]
        L.csa_ratio4_attention_workspace.restype = C.c_size_t
        L.csa_ratio4_attention_workspace.argtypes = [C.POINTER(CsaParams)]
        L.csa_ratio4_attention.restype = C.c_int
        L.csa_ratio4_attention.argtypes = [C.POINTER(CsaParams), _p]
        for name in ("csa_ratio128_compress", "csa_ratio4_main_compress",
                     "csa_ratio4_index_compress"):
            fn = getattr(L, name)
            fn.restype = C.c_int
            fn.argtypes = [C.POINTER(CompressParams), _p]
        L.csa_pool_weight.restype = C.c_int
        L.csa_pool_weight.argtypes = [_p, _p, _i64, _p]
        L.sa_check_wait_timeout.restype = C.c_int
        L.sa_check_wait_timeout.argtypes = [_p, _p, _p]
        L.sa_graph_kernel_count.restype = C.c_int
        L.sa_graph_kernel_count.argtypes = [_p]
        L.paged_attn_decode_workspace.restype = C.c_size_t
        L.paged_attn_decode_workspace.argtypes = [C.POINTER(PagedParams)]
        L.sa_rope_table.restype = C.c_int
        L.sa_rope_table.argtypes = [C.POINTER(_RopeConfig), C.POINTER(RopeTable)]
        for name, params in (("paged_attn_decode", PagedParams), ("rotary_embed", RotaryParams),
                             ("paged_kv_write", KvPagesParams), ("paged_kv_read", KvPagesParams),
                             ("attn_prefill_packed", PackedParams),
                             ("attn_weights_packed", WeightsParams),
                             ("paged_kv_select", SelectParams),
                             ("paged_kv_compact", CompactParams)):
            fn = getattr(L, name)
            fn.restype = C.c_int
            fn.argtypes = [C.POINTER(params), _p]
            # the same entry for the calls below that pack their parameters as bytes
            raw = L[name]
            raw.restype = C.c_int
            raw.argtypes = [C.c_char_p, _p]
            setattr(L, name + "_bytes", raw)
        L.paged_attn_decode_weights.restype = C.c_int
        L.paged_attn_decode_weights.argtypes = [C.POINTER(PagedParams), _p, _p]
        raw = L["paged_attn_decode_weights"]
        raw.restype, raw.argtypes = C.c_int, [C.c_char_p, _p, _p]
        L.paged_attn_decode_weights_bytes = raw
        L.paged_attn_decode_weights_workspace.restype = C.c_size_t
        L.paged_attn_decode_weights_workspace.argtypes = [C.POINTER(PagedParams)]
        L.attn_weights_packed_workspace.restype = C.c_size_t
        L.attn_weights_packed_workspace.argtypes = [C.POINTER(WeightsParams)]
        _lib = L
        return _lib


class kernel_events:
    """Measurement hook: within the ``with`` block, every call of this library
    from this host thread records ``before`` / ``after`` (timing
    ``torch.cuda.Event`` objects, recorded once here so that they exist) on its
    stream around its dominant kernel; ``before.elapsed_time(after)`` is then
    that kernel's duration for the last call."""

    def __init__(self, before, after):
        self.before, self.after = before, after

    def __enter__(self):
        for ev in (self.before, self.after):
            if not ev.cuda_event:
                ev.record()
        torch.cuda.synchronize()
        _check("sa_set_kernel_events",
               load().sa_set_kernel_events(C.c_void_p(self.before.cuda_event),
                                           C.c_void_p(self.after.cuda_event)))
        return self

    def __exit__(self, *exc):
        load().sa_set_kernel_events(None, None)
        return False


def status_string(status: int) -> str:
    return load().sa_status_string(int(status)).decode()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


def _dt(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _dev(t, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(call, rc):
    if rc != 0:
        raise SAError(call, rc)


_ws_cache: dict = {}


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """A caller-owned workspace of at least ``nbytes`` (contents irrelevant)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _workspace(nbytes: int, device, workspace=None):
    """Caller-owned scratch: the given tensor, or a cached torch allocation
    per (device, stream)."""
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    key = (str(device), torch.cuda.current_stream(device).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = new_workspace(max(nbytes, 1 << 20), device)
        _ws_cache[key] = buf
    return buf, buf.numel()


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def validate_indices(idx: torch.Tensor, bound: int = 0, bound_per_batch=None, *,
                     row_status: torch.Tensor | None = None,
                     err_word: torch.Tensor | None = None, stream=None):
    """Validate ``idx`` ``[B, I, Sq, K]`` (int32/int64) on the device.

    Returns ``(row_status uint8 [B*I*Sq], err_word uint32 [1])`` device tensors;
    ``err_word`` is zeroed here unless passed in."""
    L = load()
    _dev(idx, "idx")
    B, I, Sq, K = idx.shape
    if row_status is None:
        row_status = torch.empty(B * I * Sq, dtype=torch.uint8, device=idx.device)
    if err_word is None:
        err_word = torch.zeros(1, dtype=torch.int32, device=idx.device)
    bb = _dev(bound_per_batch, "bound_per_batch")
    rc = L.validate_indices(idx.data_ptr(), int(idx.dtype == torch.int64), B, I, Sq, K, _ptr(bb),
                            int(bound), _ptr(row_status), err_word.data_ptr(), _stream(stream))
    _check("validate_indices", rc)
    return row_status, err_word


def build_present_kv(cur_k, present_k, past_k=None, cur_v=None, present_v=None, past_v=None, *,
                     write_pos=None, err_word=None, stream=None):
    """Present K/V: concat (``write_pos`` None: present = past ++ cur along the
    sequence axis, present ``[B,H,stride,D]``) or append (cur written at
    ``write_pos[b]`` of the capacity cache ``present``)."""
    L = load()
    for n, t in (("cur_k", cur_k), ("present_k", present_k), ("past_k", past_k), ("cur_v", cur_v),
                 ("present_v", present_v), ("past_v", past_v), ("write_pos", write_pos),
                 ("err_word", err_word)):
        _dev(t, n)
    B, H, Cn, D = cur_k.shape
    P = 0 if (past_k is None or write_pos is not None) else past_k.shape[2]
    rc = L.build_present_kv(_ptr(past_k), cur_k.data_ptr(), present_k.data_ptr(), _ptr(past_v),
                            _ptr(cur_v), _ptr(present_v), _dt(cur_k), B, H, P, Cn, D,
                            present_k.shape[2], _ptr(write_pos), _ptr(err_word), _stream(stream))
    _check("build_present_kv", rc)
    return present_k, present_v


def _sparse_params(q, k_cache, v_cache, idx, y, *, scale, softcap, window, kv_len, past_len,
                   causal, sink, err_word, row_status, n_rope=0, Dv=None, k_cur=None,
                   v_cur=None, write_pos=None, bias=None, options=0):
    p = SparseParams()
    B, Hq, Sq, D = q.shape
    p.q, p.y = q.data_ptr(), _ptr(y)
    p.q_dtype = _dt(q)
    if k_cache.dtype == torch.uint8:
        p.k_cache = k_cache.data_ptr()
        p.v_cache = None
        p.kv_dtype = FP8_E4M3_B64
        p.record_stride = k_cache.shape[3]
        p.n_rope = n_rope
        p.Dv = D if Dv is None else Dv
    else:
        p.k_cache, p.v_cache = k_cache.data_ptr(), _ptr(v_cache)
        p.kv_dtype = _dt(k_cache)
        p.Dv = v_cache.shape[3]
    p.Hkv, p.T = k_cache.shape[1], k_cache.shape[2]
    if idx is not None:
        p.idx = idx.data_ptr()
        p.idx_is_i64 = int(idx.dtype == torch.int64)
        p.I, p.K = idx.shape[1], idx.shape[3]
    else:
        p.idx, p.I, p.K = None, 1, 0
    p.B, p.Hq, p.Sq, p.D = B, Hq, Sq, D
    p.sink = _ptr(sink)
    p.kv_len = _ptr(kv_len)
    p.past_len = int(past_len)
    p.causal = int(bool(causal))
    p.scale = float(scale)
    p.softcap = float(softcap)
    p.window = int(window)
    p.err_word = _ptr(err_word)
    p.row_status = _ptr(row_status)
    p.k_cur, p.v_cur, p.write_pos = _ptr(k_cur), _ptr(v_cur), _ptr(write_pos)
    p.cur_len = 0 if k_cur is None else k_cur.shape[2]
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() > 4:
            raise ValueError("bias must be float32 of rank <= 4")
        p.bias, p.bias_rank = bias.data_ptr(), bias.dim()
        for r, e in enumerate(bias.shape):
            p.bias_dims[r] = e
    p.options = int(options)
    return p


def sparse_attn_decode_workspace(q, k_cache, v_cache, idx, **kw) -> int:
    p = _sparse_params(q, k_cache, v_cache, idx, None, **_sparse_defaults(kw))
    return int(load().sparse_attn_decode_workspace(C.byref(p)))


def _sparse_defaults(kw):
    d = dict(scale=0.0, softcap=0.0, window=0, kv_len=None, past_len=0, causal=False, sink=None,
             err_word=None, row_status=None, n_rope=0, Dv=None, k_cur=None, v_cur=None,
             write_pos=None, bias=None, options=0)
    d.update(kw)
    return d


def sparse_attn_decode(q, k_cache, v_cache, idx, *, y=None, workspace=None, stream=None, **kw):
    """Selected-token attention.  ``q [B,Hq,Sq,D]``; dense cache
    ``k_cache/v_cache [B,Hkv,T,D]`` (same dtype as q) or FP8 hybrid records
    ``k_cache uint8 [B,Hkv,T,record_stride]`` (``v_cache`` None, pass
    ``n_rope``); ``idx [B,I,Sq,K]`` int32/int64.  Keyword options: scale,
    softcap, window, kv_len (int64 [B]), past_len, causal, sink (float32
    [Hq]), err_word (int32 [1], caller-zeroed), row_status (uint8 [B*I*Sq]),
    n_rope, Dv, the fused append k_cur / v_cur ([B,Hkv,C,D]) with
    write_pos (int64 [B], default T - C), bias (float32, rank <= 4,
    broadcast against [B,Hq,Sq,T]: added to the score of cache position j)
    and options (OPT_* bits).  Returns ``y [B,Hq,Sq,Dv]``."""
    L = load()
    kw = _sparse_defaults(kw)
    for n, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("idx", idx),
                 ("kv_len", kw["kv_len"]), ("sink", kw["sink"]), ("err_word", kw["err_word"]),
                 ("row_status", kw["row_status"]), ("k_cur", kw["k_cur"]), ("v_cur", kw["v_cur"]),
                 ("write_pos", kw["write_pos"]), ("bias", kw["bias"])):
        _dev(t, n)
    B, Hq, Sq, D = q.shape
    Dv = kw["Dv"] if k_cache.dtype == torch.uint8 else v_cache.shape[3]
    if Dv is None:
        Dv = D
    if y is None:
        y = torch.empty((B, Hq, Sq, Dv), dtype=q.dtype, device=q.device)
    p = _sparse_params(q, k_cache, v_cache, idx, y, **kw)
    need = int(L.sparse_attn_decode_workspace(C.byref(p)))
    ws, nb = _workspace(need, q.device, workspace)
    p.workspace, p.workspace_bytes = _ptr(ws), nb
    _check("sparse_attn_decode", L.sparse_attn_decode(C.byref(p), _stream(stream)))
    return y


_MASK_KIND = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3, torch.bool: 4,
              torch.uint8: 4}


def _prefill_params(q, k, v, y, present_k, present_v, causal, scale, softcap, err_word=None,
                    attn_mask=None, nonpad_kv_seqlen=None):
    p = PrefillParams()
    B, Hq, S, D = q.shape
    p.q, p.k, p.v, p.y = q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(y)
    p.present_k, p.present_v = _ptr(present_k), _ptr(present_v)
    p.dtype, p.causal = _dt(q), int(bool(causal))
    p.B, p.Hq, p.Hkv, p.S, p.D = B, Hq, k.shape[1], S, D
    p.scale, p.softcap = float(scale), float(softcap)
    p.err_word = _ptr(err_word)
    if attn_mask is not None:
        if attn_mask.dtype not in _MASK_KIND or attn_mask.dim() > 4:
            raise ValueError("attn_mask: float32/float16/bfloat16/bool of rank <= 4")
        p.attn_mask, p.mask_kind = attn_mask.data_ptr(), _MASK_KIND[attn_mask.dtype]
        p.mask_rank = attn_mask.dim()
        for r, e in enumerate(attn_mask.shape):
            p.mask_dims[r] = e
    p.nonpad_kv_seqlen = _ptr(nonpad_kv_seqlen)
    return p


def attn_prefill_workspace(q, k, v, causal=True, scale=0.0, softcap=0.0, attn_mask=None,
                           nonpad_kv_seqlen=None) -> int:
    p = _prefill_params(q, k, v, None, None, None, causal, scale, softcap, None, attn_mask,
                        nonpad_kv_seqlen)
    return int(load().attn_prefill_workspace(C.byref(p)))


def attn_prefill(q, k, v, *, causal=True, scale=0.0, softcap=0.0, y=None, present_k=None,
                 present_v=None, err_word=None, workspace=None, stream=None, attn_mask=None,
                 nonpad_kv_seqlen=None):
    """Dense prefill, ``q [B,Hq,S,D]``, ``k/v [B,Hkv,S,D]``; optional exact
    present K/V copies, ``attn_mask`` (float32/float16/bfloat16/bool, rank <=
    4, broadcast against ``[B,Hq,S,S]``) and ``nonpad_kv_seqlen`` (int64
    ``[B]``).  Returns ``y``."""
    L = load()
    for n, t in (("q", q), ("k", k), ("v", v), ("present_k", present_k),
                 ("present_v", present_v), ("attn_mask", attn_mask),
                 ("nonpad_kv_seqlen", nonpad_kv_seqlen)):
        _dev(t, n)
    if y is None:
        y = torch.empty_like(q)
    p = _prefill_params(q, k, v, y, present_k, present_v, causal, scale, softcap, err_word,
                        attn_mask, nonpad_kv_seqlen)
    need = int(L.attn_prefill_workspace(C.byref(p)))
    ws, nb = _workspace(need, q.device, workspace)
    p.workspace, p.workspace_bytes = _ptr(ws), nb
    _check("attn_prefill", L.attn_prefill(C.byref(p), _stream(stream)))
    return y


def _paged_params(q, k_pool, v_pool, block_table, ctx_len, y, k_new, v_new, scale, err_word,
                  options=0):
    p = PagedParams()
    B, Hq = q.shape[0], q.shape[1]
    D = q.shape[-1]
    p.q, p.k_pool, p.v_pool = q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr()
    p.k_new, p.v_new = _ptr(k_new), _ptr(v_new)
    p.block_table, p.ctx_len, p.y = block_table.data_ptr(), ctx_len.data_ptr(), _ptr(y)
    p.dtype = _dt(q)
    if k_pool.dtype == torch.uint8:
        p.pool_format, page_tokens = FP8_E4M3_PAGE, _fp8_page_tokens(k_pool, v_pool, D)
    else:
        page_tokens = k_pool.shape[2]
    p.B, p.Hq, p.Hkv, p.D = B, Hq, k_pool.shape[1], D
    p.page_tokens, p.max_pages, p.num_pages = page_tokens, block_table.shape[1], k_pool.shape[0]
    p.scale = float(scale)
    p.err_word = _ptr(err_word)
    p.options = int(options)
    return p


def paged_attn_decode_workspace(q, k_pool, v_pool, block_table, ctx_len, scale=0.0) -> int:
    p = _paged_params(q, k_pool, v_pool, block_table, ctx_len, None, None, None, scale, None)
    return int(load().paged_attn_decode_workspace(C.byref(p)))


def paged_attn_decode_weights_workspace(q, k_pool, v_pool, block_table, ctx_len, scale=0.0) -> int:
    p = _paged_params(q, k_pool, v_pool, block_table, ctx_len, None, None, None, scale, None)
    return int(load().paged_attn_decode_weights_workspace(C.byref(p)))


def paged_attn_decode(q, k_pool, v_pool, block_table, ctx_len, *, k_new=None, v_new=None,
                      scale=0.0, err_word=None, y=None, workspace=None, stream=None,
                      options=0, weights=None):
    """Paged causal decode: ``q [B,Hq,1,D]`` (or ``[B,Hq,D]``), pools
    ``[num_pages,Hkv,page_tokens,D]`` of q's dtype, or FP8 pools (uint8
    ``[num_pages,Hkv,page_tokens*(D+1)]``, see ``new_fp8_pool``; q float16 or
    bfloat16), ``block_table int32 [B,max_pages]``, ``ctx_len int32 [B]``;
    optional ``k_new/v_new [B,Hkv,D]`` written (quantised for FP8 pools) at
    token ``ctx_len-1`` first.  Returns ``y`` shaped like ``q``.

    ``weights`` (float32 ``[num_pages,Hkv,page_tokens]``, ``new_weight_pool``): the attention
    weight that each token receives, summed over the heads of its KV head's group, is added to
    its entry, and set for the new token ``ctx_len-1``."""
    L = load()
    for n, t in (("q", q), ("k_pool", k_pool), ("v_pool", v_pool), ("block_table", block_table),
                 ("ctx_len", ctx_len), ("k_new", k_new), ("v_new", v_new),
                 ("err_word", err_word)):
        _dev(t, n)
    if block_table.dtype != torch.int32 or ctx_len.dtype != torch.int32:
        raise TypeError("block_table and ctx_len must be int32")
    if weights is not None:
        return _paged_decode_weights(L, q, k_pool, v_pool, block_table, ctx_len, k_new, v_new,
                                     scale, err_word, y, workspace, stream, options, weights)
    if k_pool.dtype == torch.uint8:
        return _paged_fp8_decode(L, q, k_pool, v_pool, block_table, ctx_len, k_new, v_new, scale,
                                 err_word, y, workspace, stream, options)
    if y is None:
        y = torch.empty_like(q)
    p = _paged_params(q, k_pool, v_pool, block_table, ctx_len, y, k_new, v_new, scale, err_word,
                      options)
    need = int(L.paged_attn_decode_workspace(C.byref(p)))
    ws, nb = _workspace(need, q.device, workspace)
    p.workspace, p.workspace_bytes = _ptr(ws), nb
    _check("paged_attn_decode", L.paged_attn_decode(C.byref(p), _stream(stream)))
    return y


def _paged_decode_device(q, k_pool, v_pool, block_table, ctx_len, k_new, v_new, err_word, y):
    """The device of a paged decode whose shapes fit."""
    shape, pool = q.shape, k_pool.shape
    B, D, Hkv = shape[0], shape[-1], pool[1]
    if not (len(shape) == 3 or (len(shape) == 4 and shape[2] == 1)):
        raise ValueError("q must be [B, Hq, 1, D] or [B, Hq, D]")
    device = _same_device(q, (k_pool, v_pool, block_table, ctx_len, k_new, v_new, err_word, y))
    _paged_shapes(B, block_table, ctx_len)
    for n, t in (("k_new", k_new), ("v_new", v_new)):
        if t is not None and (t.dtype != q.dtype or t.numel() != B * Hkv * D):
            raise ValueError(f"{n} must be [B, Hkv, D] of q's dtype")
    if y is not None and (_dev(y, "y").dtype != q.dtype or y.shape != shape):
        raise ValueError("y must be shaped and typed like q")
    return device


def _paged_decode_weights(L, q, k_pool, v_pool, block_table, ctx_len, k_new, v_new, scale, err_word,
                          y, workspace, stream, options, weights):
    device = _paged_decode_device(q, k_pool, v_pool, block_table, ctx_len, k_new, v_new, err_word, y)
    shape, pool = q.shape, k_pool.shape
    B, D, Hkv = shape[0], shape[-1], pool[1]
    if k_pool.dtype == torch.uint8:
        fmt, page_tokens = FP8_E4M3_PAGE, _fp8_page_tokens(k_pool, v_pool, D)
    else:
        if len(pool) != 4 or v_pool.shape != pool or k_pool.dtype != q.dtype or \
                v_pool.dtype != q.dtype or pool[3] != D:
            raise ValueError("pools must be [num_pages, Hkv, page_tokens, D] of q's dtype, or FP8 "
                             "pools")
        fmt, page_tokens = 0, pool[2]
    _weight_pool(weights, pool[0], Hkv, page_tokens, device)
    dtype = _dt(q)
    with _launching(device, stream) as s:
        if y is None:
            y = torch.empty_like(q)

        def params(ws, nbytes):
            return _PAGED.pack(
                q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), _addr(k_new), _addr(v_new),
                block_table.data_ptr(), ctx_len.data_ptr(), y.data_ptr(), dtype, options, B,
                shape[1], Hkv, D, page_tokens, block_table.shape[1], pool[0], scale, fmt,
                _addr(err_word), ws, nbytes)

        _call_with_workspace(
            "paged_attn_decode_weights", params, device, s, workspace,
            lambda p: L.paged_attn_decode_weights_bytes(p, weights.data_ptr(), s),
            lambda p: L.paged_attn_decode_weights_workspace(C.byref(PagedParams.from_buffer_copy(p))))
    return y


def _call_with_workspace(name, params, device, s, workspace, call, size):
    """Run ``call`` on parameters with the given workspace, the kept one, or one of ``size``."""
    if workspace is None:
        # the kept scratch is nearly always large enough: ask only when it is not
        ws = _kept_workspace(device, s)
        if ws is not None:
            rc = call(params(ws.data_ptr(), ws.numel()))
            if rc != ERR_WORKSPACE:
                _check(name, rc)
                return
    ws, nb = _stream_workspace(int(size(params(0, 0))), device, s, workspace)
    _check(name, call(params(_addr(ws), nb)))


def _paged_fp8_decode(L, q, k_pool, v_pool, block_table, ctx_len, k_new, v_new, scale, err_word,
                      y, workspace, stream, options):
    device = _paged_decode_device(q, k_pool, v_pool, block_table, ctx_len, k_new, v_new, err_word, y)
    shape, pool = q.shape, k_pool.shape
    B, D, Hkv = shape[0], shape[-1], pool[1]
    page_tokens, dtype = _fp8_page_tokens(k_pool, v_pool, D), _dt(q)
    with _launching(device, stream) as s:
        if y is None:
            y = torch.empty_like(q)

        def params(ws, nbytes):
            return _PAGED.pack(
                q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), _addr(k_new), _addr(v_new),
                block_table.data_ptr(), ctx_len.data_ptr(), y.data_ptr(), dtype, options, B,
                shape[1], Hkv, D, page_tokens, block_table.shape[1], pool[0], scale,
                FP8_E4M3_PAGE, _addr(err_word), ws, nbytes)

        if workspace is None:
            # the kept scratch is nearly always large enough: ask only when it is not
            ws = _kept_workspace(device, s)
            if ws is not None:
                rc = L.paged_attn_decode_bytes(params(ws.data_ptr(), ws.numel()), s)
                if rc != ERR_WORKSPACE:
                    _check("paged_attn_decode", rc)
                    return y
        p = PagedParams.from_buffer_copy(params(0, 0))
        ws, nb = _stream_workspace(int(L.paged_attn_decode_workspace(C.byref(p))), device, s,
                                   workspace)
        _check("paged_attn_decode", L.paged_attn_decode_bytes(params(_addr(ws), nb), s))
    return y


def sparse_attn_decode_noalloc(q, k_cache, v_cache, idx, *, y=None, stream=None, **kw):
    """``sparse_attn_decode`` without caller-provided scratch: the library's
    built-in device buffer (``NOALLOC_SCRATCH_BYTES``) serves every call, so
    calls must not overlap on the GPU.  Same arguments, minus ``workspace``."""
    L = load()
    kw = _sparse_defaults(kw)
    for n, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("idx", idx),
                 ("kv_len", kw["kv_len"]), ("sink", kw["sink"]), ("err_word", kw["err_word"]),
                 ("row_status", kw["row_status"]), ("k_cur", kw["k_cur"]), ("v_cur", kw["v_cur"]),
                 ("write_pos", kw["write_pos"]), ("bias", kw["bias"])):
        _dev(t, n)
    B, Hq, Sq, D = q.shape
    Dv = kw["Dv"] if k_cache.dtype == torch.uint8 else v_cache.shape[3]
    if Dv is None:
        Dv = D
    if y is None:
        y = torch.empty((B, Hq, Sq, Dv), dtype=q.dtype, device=q.device)
    p = _sparse_params(q, k_cache, v_cache, idx, y, **kw)
    _check("sparse_attn_decode_noalloc", L.sparse_attn_decode_noalloc(C.byref(p), _stream(stream)))
    return y


def _index_params(query, weight, keys, selected, *, topk, query_start, query_start_b,
                  out_heads, ascending, row_status, err_word):
    p = IndexSelectParams()
    B, S, IH, ID = query.shape
    p.query, p.weight, p.keys = query.data_ptr(), weight.data_ptr(), keys.data_ptr()
    p.selected = _ptr(selected)
    p.row_status, p.err_word = _ptr(row_status), _ptr(err_word)
    p.B, p.S, p.IH, p.ID = B, S, IH, ID
    p.R, p.key_stride = keys.shape[1], keys.shape[2]
    p.topk, p.out_heads = int(topk), int(out_heads)
    p.query_start = int(query_start)
    p.query_start_b = _ptr(query_start_b)
    p.ascending = int(bool(ascending))
    return p


def sparse_index_select_workspace(query, weight, keys, *, topk, out_heads=1) -> int:
    p = _index_params(query, weight, keys, None, topk=topk, query_start=0, query_start_b=None,
                      out_heads=out_heads, ascending=False, row_status=None, err_word=None)
    return int(load().sparse_index_select_workspace(C.byref(p)))


def sparse_index_select(query, weight, keys, *, topk, query_start=0, query_start_b=None,
                        out_heads=1, ascending=False, row_status=None, err_word=None,
                        selected=None, workspace=None, stream=None):
    """Ratio-4 index scoring and top-k selection.  ``query`` float32
    ``[B, S, IH, ID]``, ``weight`` float32 ``[B, S, IH]``, ``keys`` uint8
    ``[B, R, key_stride]`` FP4 records; query s of batch b sits at position
    ``query_start + s`` (or ``query_start_b[b] + s``, int64 ``[B]``).
    Returns ``selected`` int32 ``[B, out_heads, S, topk]`` (score order, or
    ascending records with ``ascending``), -1 past the causal records;
    ``row_status`` (uint8 ``[B*S]``) / ``err_word`` receive the tie and
    non-finite flags."""
    L = load()
    for n, t in (("query", query), ("weight", weight), ("keys", keys),
                 ("query_start_b", query_start_b), ("row_status", row_status),
                 ("err_word", err_word), ("selected", selected)):
        _dev(t, n)
    if query.dtype != torch.float32 or weight.dtype != torch.float32 or keys.dtype != torch.uint8:
        raise TypeError("query and weight must be float32, keys uint8")
    B, S = query.shape[0], query.shape[1]
    if selected is None:
        selected = torch.empty((B, out_heads, S, topk), dtype=torch.int32, device=query.device)
    p = _index_params(query, weight, keys, selected, topk=topk, query_start=query_start,
                      query_start_b=query_start_b, out_heads=out_heads, ascending=ascending,
                      row_status=row_status, err_word=err_word)
    need = int(L.sparse_index_select_workspace(C.byref(p)))
    ws, nb = _workspace(need, query.device, workspace)
    p.workspace, p.workspace_bytes = _ptr(ws), nb
    _check("sparse_index_select", L.sparse_index_select(C.byref(p), _stream(stream)))
    return selected


def _csa_params(query, current_kv, records, selected, y, *, total, n_rope, scale, sink, bias,
                err_word):
    p = CsaParams()
    B, S, H, D = query.shape
    p.query, p.current_kv = query.data_ptr(), _ptr(current_kv)
    p.records, p.selected, p.y = records.data_ptr(), selected.data_ptr(), _ptr(y)
    p.sink, p.err_word = _ptr(sink), _ptr(err_word)
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() > 4:
            raise ValueError("bias must be float32 of rank <= 4")
        p.bias, p.bias_rank = bias.data_ptr(), bias.dim()
        for r, e in enumerate(bias.shape):
            p.bias_dims[r] = e
    p.q_dtype = _dt(query)
    p.kv_dtype = _dt(current_kv) if current_kv is not None else _dt(query)
    p.B, p.S, p.H, p.D = B, S, H, D
    p.n_rope = int(n_rope)
    p.L = current_kv.shape[1] if current_kv is not None else 0
    p.R, p.record_stride = records.shape[1], records.shape[2]
    p.topk, p.total, p.scale = selected.shape[2], int(total), float(scale)
    return p


def csa_ratio4_attention_workspace(query, current_kv, records, selected, *, total, n_rope,
                                   scale=0.0, sink=None, bias=None) -> int:
    p = _csa_params(query, current_kv, records, selected, None, total=total, n_rope=n_rope,
                    scale=scale, sink=sink, bias=bias, err_word=None)
    return int(load().csa_ratio4_attention_workspace(C.byref(p)))


def csa_ratio4_attention(query, current_kv, records, selected, *, total, n_rope, scale=0.0,
                         sink=None, bias=None, err_word=None, y=None, workspace=None,
                         stream=None):
    """Compressed sparse attention, ratio 4, in the pages' own form.  ``query``
    ``[B, S, H, D]`` (float32 / bfloat16), ``current_kv`` ``[B, L, D]``,
    ``records`` uint8 ``[B, R, record_stride]`` hybrid FP8, ``selected`` int32
    ``[B, S, topk]``; ``total`` tokens so far; optional ``sink`` float32 ``[H]``
    and ``bias`` float32 (rank <= 4, against ``[B, H, S, candidates]``).
    Returns ``y`` shaped and typed like ``query``."""
    L = load()
    for n, t in (("query", query), ("current_kv", current_kv), ("records", records),
                 ("selected", selected), ("sink", sink), ("bias", bias), ("err_word", err_word)):
        _dev(t, n)
    if selected.dtype != torch.int32 or records.dtype != torch.uint8:
        raise TypeError("selected must be int32 and records uint8")
    if y is None:
        y = torch.empty_like(query)
    p = _csa_params(query, current_kv, records, selected, y, total=total, n_rope=n_rope,
                    scale=scale, sink=sink, bias=bias, err_word=err_word)
    need = int(L.csa_ratio4_attention_workspace(C.byref(p)))
    ws, nb = _workspace(need, query.device, workspace)
    p.workspace, p.workspace_bytes = _ptr(ws), nb
    _check("csa_ratio4_attention", L.csa_ratio4_attention(C.byref(p), _stream(stream)))
    return y


# ---- CSA compression stages ---------------------------------------------------------------

def _compress(name, ratio, D, kv, gate, ape, norm, carry, *, n_rope, total, records, logical,
              err_word, stream):
    L = load()
    for n, t in (("kv", kv), ("gate", gate), ("ape", ape), ("norm", norm), ("carry", carry),
                 ("records", records), ("logical", logical), ("err_word", err_word)):
        _dev(t, n)
    for n, t in (("kv", kv), ("gate", gate), ("ape", ape), ("norm", norm), ("carry", carry),
                 ("logical", logical)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise TypeError(f"{n} must be a contiguous float32 tensor")
    if records is not None and (records.dtype != torch.uint8 or not records.is_contiguous()):
        raise TypeError("records must be a contiguous uint8 tensor")
    B, S = kv.shape[0], kv.shape[1]
    p = CompressParams()
    p.kv, p.gate, p.ape, p.norm = kv.data_ptr(), gate.data_ptr(), ape.data_ptr(), norm.data_ptr()
    p.carry, p.records, p.logical = carry.data_ptr(), _ptr(records), _ptr(logical)
    p.err_word = _ptr(err_word)
    p.B, p.S, p.D, p.n_rope, p.total = B, S, D, int(n_rope), int(total)
    if records is not None:
        p.rows, p.record_stride = records.shape[1], records.shape[2]
    else:
        p.rows, p.record_stride = logical.shape[1], 0
    _check(name, getattr(L, name)(C.byref(p), _stream(stream)))


def csa_ratio128_compress(kv, gate, ape, norm, carry, *, n_rope, total, records=None,
                          logical=None, err_word=None, stream=None):
    """Append ``S`` tokens to a ratio-128 compression stream.  ``kv``, ``gate``
    float32 ``[B, S, D]``, ``ape`` ``[128, D]``, ``norm`` ``[D]``, ``carry``
    ``[B, 128, 2, D]`` (updated in place); every block of 128 tokens that
    closes is written to ``records`` (uint8 ``[B, rows, stride]``, hybrid
    FP8) and/or ``logical`` (float32 ``[B, rows, D]``) at row ``p // 128``."""
    _compress("csa_ratio128_compress", 128, kv.shape[2], kv, gate, ape, norm, carry,
              n_rope=n_rope, total=total, records=records, logical=logical,
              err_word=err_word, stream=stream)


def csa_ratio4_main_compress(kv, gate, ape, norm, carry, *, n_rope, total, records=None,
                             logical=None, err_word=None, stream=None):
    """Append ``S`` tokens to a ratio-4 attention-record stream.  ``kv``,
    ``gate`` float32 ``[B, S, 2D]``, ``ape`` ``[4, 2D]``, ``norm`` ``[D]``,
    ``carry`` ``[B, 8, 2, 2D]`` (updated in place); records as for ratio 128,
    at row ``p // 4``."""
    _compress("csa_ratio4_main_compress", 4, kv.shape[2] // 2, kv, gate, ape, norm, carry,
              n_rope=n_rope, total=total, records=records, logical=logical,
              err_word=err_word, stream=stream)


def csa_ratio4_index_compress(kv, gate, ape, norm, carry, *, n_rope, total, records=None,
                              logical=None, err_word=None, stream=None):
    """Append ``S`` tokens to a ratio-4 index-key stream (FP4 keys of
    ``D / 32 * 17`` bytes, Hadamard-transformed); shapes as for
    ``csa_ratio4_main_compress``."""
    _compress("csa_ratio4_index_compress", 4, kv.shape[2] // 2, kv, gate, ape, norm, carry,
              n_rope=n_rope, total=total, records=records, logical=logical,
              err_word=err_word, stream=stream)


def graph_kernel_count(graph) -> int:
    """Kernel nodes in a captured ``torch.cuda.CUDAGraph`` (measurement hook:
    how many kernels one captured call launches)."""
    n = load().sa_graph_kernel_count(C.c_void_p(graph.raw_cuda_graph()))
    _check("sa_graph_kernel_count", min(n, 0))
    return n


def check_wait_timeout(device="cuda", stream=None):
    """Runs the library's bounded-wait timeout path once (one warp waits on a
    barrier nothing arrives on, about a second); returns ``(err_word, out)``,
    int32 CUDA tensors of 1 and 4 entries (see ``sa_check_wait_timeout``)."""
    err = torch.zeros(1, dtype=torch.int32, device=device)
    out = torch.zeros(4, dtype=torch.int32, device=device)
    _check("sa_check_wait_timeout",
           load().sa_check_wait_timeout(err.data_ptr(), out.data_ptr(), _stream(stream)))
    return err, out


def csa_pool_weight(t, *, w=None, stream=None):
    """``e^t`` rounded to binary32 as the compression pool computes it;
    ``t`` a contiguous float32 CUDA tensor."""
    _dev(t, "t")
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError("t must be a contiguous float32 tensor")
    if w is None:
        w = torch.empty_like(t)
    _check("csa_pool_weight", load().csa_pool_weight(t.data_ptr(), w.data_ptr(), t.numel(),
                                                      _stream(stream)))
    return w


# ---- the serving step around a paged cache --------------------------------------------------

def _stream_handle(index):
    """The current stream's handle on a device.  (``current_stream()`` builds a Stream
    object first, which takes as long as the launch.)"""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


class _launching:
    """The tensors' device made current and the launching stream's handle:
    ``stream``'s, or the device's current one's.  Tensors allocated inside belong
    to that stream."""

    __slots__ = ("device", "stream", "stack")

    def __init__(self, device, stream):
        self.device, self.stream, self.stack = device, stream, None

    def __enter__(self):
        index = self.device.index
        if self.stream is not None and self.stream.device != self.device:
            raise ValueError(f"stream is on {self.stream.device}, the tensors are on {self.device}")
        if self.stream is None and index == torch.cuda.current_device():
            return _stream_handle(index)
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(self.device))
        if self.stream is None:
            return _stream_handle(index)
        self.stack.enter_context(torch.cuda.stream(self.stream))
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


class _Kept(threading.local):
    """Scratch kept per host thread, device and stream (a handle).  Per thread, as a call is
    several launches: two threads' launches on one stream may alternate."""

    def __init__(self):
        self.of = {}


_kept = _Kept()


def _kept_workspace(device, stream):
    """The scratch kept for this thread's calls on ``stream`` (a handle), or None: none
    yet, or a graph is being captured."""
    ws = _kept.of.get((device.index, stream))
    return None if ws is None or torch.cuda.is_current_stream_capturing() else ws


def _stream_workspace(nbytes, device, stream, workspace):
    """Scratch for one call on ``stream`` (a handle): the given tensor, else one
    kept per (thread, device, stream), so that calls that may overlap never share it.
    Under graph capture it comes from the graph's own memory instead: a kept
    tensor could be replaced while the graph still names it, or be shared with
    another graph that replays at the same time."""
    if workspace is not None:
        if _dev(workspace, "workspace").device != device:
            raise ValueError(f"workspace is on {workspace.device}, not on {device}")
        return workspace, workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, 0
    if torch.cuda.is_current_stream_capturing():
        return new_workspace(nbytes, device), nbytes
    key = (device.index, stream)
    buf = _kept.of.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = new_workspace(max(nbytes, 1 << 20), device)
        _kept.of[key] = buf
    return buf, buf.numel()


def _rows(t, name, dtype=None, dims=3):
    """The shape and strides of a CUDA tensor whose last axis is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    shape, strides = t.shape, t.stride()
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} axes")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    return shape, strides


def _same_device(first, others):
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on {t.device}, not on {device}")
    return device


def _int32(t, name, numel=None):
    _dev(t, name)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries")
    return t


def _paged_shapes(B, block_table, ctx_len):
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    if ctx_len.numel() != B:
        raise ValueError("ctx_len must be [B]")


def _fp8_page_tokens(k_pool, v_pool, D):
    """Tokens of a page of the FP8 pools (uint8 [num_pages, Hkv, page_tokens * (D + 1)])."""
    if k_pool.dim() != 3 or v_pool.shape != k_pool.shape or v_pool.dtype != torch.uint8:
        raise ValueError("FP8 pools are two uint8 tensors [num_pages, Hkv, page_tokens * (D + 1)]")
    if k_pool.shape[2] % (D + 1):
        raise ValueError(f"the pools' pages do not hold rows of {D} codes and a scale")
    return k_pool.shape[2] // (D + 1)


def new_fp8_pool(num_pages: int, Hkv: int, page_tokens: int, D: int, device="cuda") -> torch.Tensor:
    """A zeroed FP8 page pool, uint8 ``[num_pages, Hkv, page_tokens * (D + 1)]``: per page and
    head ``page_tokens`` rows of D E4M3 codes, then their E8M0 scale bytes."""
    return torch.zeros((num_pages, Hkv, page_tokens * (D + 1)), dtype=torch.uint8, device=device)


_SCALING = {"none": 0, "linear": 1, "ntk": 2, "ramp": 3}


def rope_table(rotary_dim, *, base=10000.0, interleaved=False, scaling="none", factor=1.0,
               original_len=0, ramp=(1.0, 32.0), mscale=1.0, inv_freq=None) -> RopeTable:
    """The angles of ``rotary_dim // 2`` rotary pairs, computed once in 64 bits on the host.

    Pair i turns by ``position * f_i``, ``f_i = base ** (-2i / rotary_dim)``, scaled for long
    contexts: ``"linear"`` (f / factor), ``"ntk"`` (a larger base) or ``"ramp"`` (pairs with more
    than ``ramp[1]`` turns over ``original_len`` tokens keep f, those with fewer than ``ramp[0]``
    take f / factor, a linear mix between); or ``inv_freq`` gives the f_i.  ``mscale`` multiplies
    the rotated dims.  ``interleaved`` pairs dims (2i, 2i + 1), otherwise (i, i + rotary_dim / 2)."""
    c = _RopeConfig()
    c.rotary_dim, c.interleaved, c.mscale = int(rotary_dim), int(bool(interleaved)), float(mscale)
    if inv_freq is not None:
        freqs = [float(f) for f in inv_freq]
        if len(freqs) != c.rotary_dim // 2:
            raise ValueError("inv_freq must have rotary_dim / 2 entries")
        keep = (C.c_double * len(freqs))(*freqs)
        c.scaling, c.inv_freq = 4, C.cast(keep, _p)
    else:
        if scaling not in _SCALING:
            raise ValueError(f"scaling must be one of {sorted(_SCALING)}")
        c.scaling = _SCALING[scaling]
    c.base, c.factor, c.original_len = float(base), float(factor), float(original_len)
    c.ramp_low, c.ramp_high = float(ramp[0]), float(ramp[1])
    out = RopeTable()
    _check("rope_table", load().sa_rope_table(C.byref(c), C.byref(out)))
    return out


def _rope_arg(rope):
    if rope is None:
        return None
    if not isinstance(rope, RopeTable):
        raise TypeError("rope must come from rope_table()")
    return C.addressof(rope)


def rotary_embed(q, k, positions, rope, *, q_out=None, k_out=None, stream=None):
    """Rotary positions of ``q`` and ``k`` (or ``k`` None) in one launch.

    Packed tensors ``[T, H, D]`` with ``positions`` int32/int64 ``[T]``, or head-major ones
    ``[B, H, S, D]`` with positions ``[S]`` (every batch) or ``[B, S]``; only the last axis has to
    be contiguous, so views into a fused projection are fine.  ``rope`` comes from
    ``rope_table``.  ``q_out`` / ``k_out`` may be the inputs themselves.  Returns
    ``(q_out, k_out)``."""
    L = load()
    dims = 4 if isinstance(q, torch.Tensor) and q.dim() == 4 else 3
    qs, qst = _rows(q, "q", dims=dims)
    dtype = _dt(q)
    _dev(positions, "positions")
    i64 = positions.dtype == torch.int64
    if not i64 and positions.dtype != torch.int32:
        raise TypeError("positions must be int32 or int64")
    ps = tuple(positions.shape)
    if dims == 3:
        B, (S, Hq, D) = 1, qs
        if ps != (S,):
            raise ValueError("positions must be [T]")
    else:
        B, Hq, S, D = qs
        if ps != (S,) and ps != (B, S):
            raise ValueError("positions must be [S] or [B, S]")
    Hk, kst = 0, None
    if k is not None:
        ks, kst = _rows(k, "k", q.dtype, dims)
        if ks[0] != qs[0] or ks[-1] != D or (dims == 4 and ks[2] != S):
            raise ValueError("q and k must have the same tokens and head size")
        Hk = ks[1]
    elif k_out is not None:
        raise ValueError("k_out needs k")
    device = _same_device(q, (k, positions, q_out, k_out))
    for n, t, o in (("q_out", q, q_out), ("k_out", k, k_out)):
        if o is not None and _rows(o, n, q.dtype, dims)[0] != t.shape:
            raise ValueError(f"{n} must be shaped like its input")
    with _launching(device, stream) as s:
        if q_out is None:
            q_out = torch.empty(qs, dtype=q.dtype, device=device)
        if k is not None and k_out is None:
            k_out = torch.empty(ks, dtype=q.dtype, device=device)
        table = _rope_arg(rope)
        if S * B * D * max(Hq, Hk) == 0:  # (keys without queries go on, and are refused)
            return q_out, k_out
        token, head = (0, 1) if dims == 3 else (2, 1)
        strides = []
        for st in (qst, kst, q_out.stride(), k_out.stride() if Hk else None):
            strides += (0, 0, 0) if st is None else (st[0] if dims == 4 else 0, st[token], st[head])
        p = _ROTARY.pack(
            q.data_ptr(), _addr(k), q_out.data_ptr(), _addr(k_out), positions.data_ptr(), table,
            dtype, i64, B, S, Hq, Hk, D, S if len(ps) == 2 else 0, *strides)
        _check("rotary_embed", L.rotary_embed_bytes(p, s))
    return q_out, k_out


def _kv_pages_params(k, v, k_pool, v_pool, block_table, ctx_len, seq_start, rope, err_word):
    """(packed parameters, device) of a page write or read-back; None for no rows."""
    shape, kst = _rows(k, "k")
    vshape, vst = _rows(v, "v", k.dtype)
    if vshape != shape:
        raise ValueError("k and v must have the same shape")
    _dev(k_pool, "k_pool")
    _dev(v_pool, "v_pool")
    _dev(err_word, "err_word")
    _int32(block_table, "block_table")
    _int32(ctx_len, "ctx_len")
    B = ctx_len.numel()
    _paged_shapes(B, block_table, ctx_len)
    if seq_start is not None:
        _int32(seq_start, "seq_start", B + 1)
    device = _same_device(k, (v, k_pool, v_pool, block_table, ctx_len, seq_start, err_word))
    T, Hkv, D = shape
    pool = k_pool.shape
    if k_pool.dtype == torch.uint8:
        fmt, page_tokens = FP8_E4M3_PAGE, _fp8_page_tokens(k_pool, v_pool, D)
    else:
        if len(pool) != 4 or k_pool.dtype != k.dtype or v_pool.dtype != k.dtype or \
                v_pool.shape != pool or pool[3] != D:
            raise ValueError("pools must be [num_pages, Hkv, page_tokens, D] of the rows' dtype, "
                             "or FP8 pools")
        fmt, page_tokens = 0, pool[2]
    if pool[1] != Hkv:
        raise ValueError("the pools and the rows have different head counts")
    if seq_start is None and T != B:
        raise ValueError("without seq_start every sequence has one row")
    dtype, table = _dt(k), _rope_arg(rope)
    if T * Hkv * D == 0:
        return None, device
    return _KV_PAGES.pack(
        k.data_ptr(), v.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
        ctx_len.data_ptr(), _addr(seq_start), table or 0, _addr(err_word), dtype, fmt, T, B,
        Hkv, D, page_tokens, block_table.shape[1], pool[0], kst[0], kst[1], vst[0],
        vst[1]), device


def paged_kv_write(k, v, k_pool, v_pool, block_table, ctx_len, seq_start=None, *, rope=None,
                   err_word=None, stream=None):
    """Write new tokens' K and V into their pages, K rotated first when ``rope`` (from
    ``rope_table``) is given, both quantised when the pools are FP8 (``new_fp8_pool``).

    ``k/v [T, Hkv, D]`` packed rows (only the last axis contiguous): sequence b owns rows
    ``seq_start[b] .. seq_start[b+1]`` (int32 ``[B+1]``; None: one row each), the last tokens of
    its ``ctx_len[b]`` (int32 ``[B]``, the new tokens counted)."""
    L = load()
    p, device = _kv_pages_params(k, v, k_pool, v_pool, block_table, ctx_len, seq_start, rope,
                                 err_word)
    if p is None:
        return
    with _launching(device, stream) as s:
        _check("paged_kv_write", L.paged_kv_write_bytes(p, s))


def paged_kv_read(k_pool, v_pool, block_table, ctx_len, seq_start, k=None, v=None, *, total=None,
                  head_dim=None, dtype=torch.bfloat16, err_word=None, stream=None):
    """Read contexts back from their pages into packed rows ``k/v [T, Hkv, D]``: row
    ``seq_start[b] + i`` receives token i of sequence b (dequantised from FP8 pools and rounded
    once).  ``k`` and ``v`` are given, or allocated as ``[total, Hkv, head_dim]`` of ``dtype``
    (zeros, so that rows of no sequence are defined).  Returns ``(k, v)``."""
    L = load()
    _dev(k_pool, "k_pool")
    if (k is None) != (v is None):
        raise ValueError("give both k and v, or neither")
    with _launching(k_pool.device, stream) as s:
        if k is None:
            if total is None or head_dim is None:
                raise ValueError("give k and v, or total and head_dim")
            shape = (int(total), k_pool.shape[1], int(head_dim))
            k = torch.zeros(shape, dtype=dtype, device=k_pool.device)
            v = torch.zeros(shape, dtype=dtype, device=k_pool.device)
        if seq_start is None:
            raise ValueError("seq_start is required")
        p, _ = _kv_pages_params(k, v, k_pool, v_pool, block_table, ctx_len, seq_start, None,
                                err_word)
        if p is not None:
            _check("paged_kv_read", L.paged_kv_read_bytes(p, s))
    return k, v


def attn_prefill_packed(q, k, v, q_start, k_start=None, *, causal=True, scale=0.0, softcap=0.0,
                        y=None, err_word=None, stream=None):
    """Prefill attention over packed sequences of different lengths: ``q [Tq, Hq, D]``,
    ``k/v [Tk, Hkv, D]`` (only the last axis contiguous), sequence b's query rows at
    ``q_start[b] .. q_start[b+1]`` and its key rows at ``k_start[b] ..`` (int32 ``[B+1]``;
    ``k_start`` None: ``q_start``).  With more keys than queries the queries are the last tokens
    of the context (causal: query i sees keys ``<= i + nk - nq``); a query that sees no key gives
    0.  Rows behind the last sequence are not written.  Returns ``y [Tq, Hq, D]``."""
    L = load()
    qs, qst = _rows(q, "q")
    ks, kst = _rows(k, "k", q.dtype)
    vs, vst = _rows(v, "v", q.dtype)
    Tq, Hq, D = qs
    Tk, Hkv, _ = ks
    if vs != ks or ks[2] != D:
        raise ValueError("k and v must have the same shape, and q's head size")
    _int32(q_start, "q_start")
    B = q_start.numel() - 1
    if k_start is not None:
        _int32(k_start, "k_start", B + 1)
    elif Tk != Tq:
        raise ValueError("k_start is required when q and k have different rows")
    _dev(err_word, "err_word")
    device = _same_device(q, (k, v, q_start, k_start, err_word, y))
    if y is not None and _rows(y, "y", q.dtype)[0] != qs:
        raise ValueError("y must be shaped like q")
    with _launching(device, stream) as s:
        if y is None:
            y = torch.empty(qs, dtype=q.dtype, device=device)
        if Tq * Hq * D == 0:
            return y
        if Tk == 0:  # no keys anywhere: an empty tensor has no address to give
            k = v = torch.empty((1, Hkv, D), dtype=q.dtype, device=device)
            kst = vst = k.stride()
        yst = y.stride()
        p = _PACKED.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), y.data_ptr(), q_start.data_ptr(),
            _addr(k_start), _addr(err_word), _dt(q), bool(causal), B, Tq, Tk, Hq, Hkv, D,
            qst[0], qst[1], kst[0], kst[1], vst[0], vst[1], yst[0], yst[1], scale, softcap)
        _check("attn_prefill_packed", L.attn_prefill_packed_bytes(p, s))
    return y


# ---- cache eviction by accumulated attention weight -------------------------------------------

def new_weight_pool(num_pages: int, Hkv: int, page_tokens: int, device="cuda") -> torch.Tensor:
    """A pool of attention weights, zeroed: float32 ``[num_pages, Hkv, page_tokens]``, addressed
    like the pages of K and V."""
    return torch.zeros((num_pages, Hkv, page_tokens), dtype=torch.float32, device=device)


def _weight_pool(weights, num_pages, Hkv, page_tokens, device):
    _dev(weights, "weights")
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if tuple(weights.shape) != (num_pages, Hkv, page_tokens):
        raise ValueError(f"weights must be [{num_pages}, {Hkv}, {page_tokens}]")
    if weights.device != device:
        raise ValueError(f"weights are on {weights.device}, not on {device}")


def attn_weights_packed(q, k, weights, block_table, q_start, k_start=None, *, scale=0.0,
                        accumulate=True, err_word=None, workspace=None, stream=None):
    """The attention weight that each key receives from packed queries, into a weights pool.

    ``q [Tq, Hq, D]``, ``k [Tk, Hkv, D]`` and the starts as for ``attn_prefill_packed`` (causal: a
    sequence's queries are the last tokens of its keys).  Token j's weight in head h of
    ``weights`` (float32 ``[num_pages, Hkv, page_tokens]``, through ``block_table`` int32
    ``[B, max_pages]``) becomes the sum of the probabilities that the queries of the head's group
    give it: set for the queries' own tokens, added to the others', or set for all with
    ``accumulate=False`` (of a page that two sequences share, to those of either).  The scores
    have no softcap.  Returns ``weights``."""
    L = load()
    qs, qst = _rows(q, "q")
    ks, kst = _rows(k, "k", q.dtype)
    Tq, Hq, D = qs
    Tk, Hkv, _ = ks
    if ks[2] != D:
        raise ValueError("q and k must have the same head size")
    _int32(q_start, "q_start")
    B = q_start.numel() - 1
    if k_start is not None:
        _int32(k_start, "k_start", B + 1)
    elif Tk != Tq:
        raise ValueError("k_start is required when q and k have different rows")
    _int32(block_table, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _dev(err_word, "err_word")
    device = _same_device(q, (k, block_table, q_start, k_start, err_word))
    if _dev(weights, "weights").dim() != 3:
        raise ValueError("weights must be [num_pages, Hkv, page_tokens]")
    _weight_pool(weights, weights.shape[0], Hkv, weights.shape[2], device)
    dtype = _dt(q)
    with _launching(device, stream) as s:
        if Tq * Tk * Hq * Hkv * D == 0:
            return weights

        def params(ws, nbytes):
            return _WEIGHTS.pack(
                q.data_ptr(), k.data_ptr(), weights.data_ptr(), block_table.data_ptr(),
                q_start.data_ptr(), _addr(k_start), _addr(err_word), dtype, bool(accumulate), B,
                Tq, Tk, Hq, Hkv, D, weights.shape[2], block_table.shape[1], weights.shape[0],
                qst[0], qst[1], kst[0], kst[1], scale, 0, ws, nbytes)

        _call_with_workspace(
            "attn_weights_packed", params, device, s, workspace,
            lambda p: L.attn_weights_packed_bytes(p, s),
            lambda p: L.attn_weights_packed_workspace(C.byref(WeightsParams.from_buffer_copy(p))))
    return weights


def paged_kv_select(weights, block_table, ctx_len, budget, *, sink=0, recent=0, keep=None,
                    new_len=None, err_word=None, stream=None):
    """The tokens that each KV head keeps of contexts that have outgrown ``budget`` tokens: the
    first ``sink``, the last ``recent``, and of those between them the ones with the largest
    accumulated weights (ties: the lower token; NaN counts as -inf); all of a shorter context.

    ``weights`` float32 ``[num_pages, Hkv, page_tokens]``, ``block_table`` int32 ``[B, max_pages]``,
    ``ctx_len`` int32 ``[B]``.  Returns ``(keep, new_len)``: int32 ``[B, Hkv, budget]``, ascending,
    -1 behind the last, and int32 ``[B]``, ``min(ctx_len, budget)``."""
    L = load()
    _dev(weights, "weights")
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if weights.dim() != 3:
        raise ValueError("weights must be [num_pages, Hkv, page_tokens]")
    _int32(block_table, "block_table")
    _int32(ctx_len, "ctx_len")
    _dev(err_word, "err_word")
    B = ctx_len.numel()
    _paged_shapes(B, block_table, ctx_len)
    num_pages, Hkv, page_tokens = weights.shape
    budget = int(budget)
    device = _same_device(weights, (block_table, ctx_len, keep, new_len, err_word))
    if keep is not None:
        _int32(keep, "keep", B * Hkv * budget)
    if new_len is not None:
        _int32(new_len, "new_len", B)
    with _launching(device, stream) as s:
        if keep is None:
            keep = torch.empty((B, Hkv, max(budget, 0)), dtype=torch.int32, device=device)
        if new_len is None:
            new_len = torch.empty(B, dtype=torch.int32, device=device)
        p = _SELECT.pack(weights.data_ptr(), block_table.data_ptr(), ctx_len.data_ptr(),
                         keep.data_ptr(), new_len.data_ptr(), _addr(err_word), B, Hkv, page_tokens,
                         block_table.shape[1], num_pages, budget, int(sink), int(recent))
        _check("paged_kv_select", L.paged_kv_select_bytes(p, s))
    return keep, new_len


def paged_kv_compact(k_pool, v_pool, block_table, ctx_len, keep, *, weights=None, head_dim=None,
                     err_word=None, stream=None):
    """Move the kept rows to the front of their sequences' pages, in place: token i of sequence b
    and KV head h becomes token ``keep[b, h, i]`` (its rows of K and V and its weight).

    ``keep`` int32 ``[B, Hkv, width]``, ascending, -1 behind the last, as ``paged_kv_select`` returns
    it; ``ctx_len`` int32 ``[B]``, the lengths before.  FP8 pools need ``weights`` or ``head_dim``
    to tell their rows' size.  A sequence's pages must be its own."""
    L = load()
    for n, t in (("k_pool", k_pool), ("v_pool", v_pool), ("err_word", err_word)):
        _dev(t, n)
    _int32(block_table, "block_table")
    _int32(ctx_len, "ctx_len")
    _int32(keep, "keep")
    B, pool = ctx_len.numel(), k_pool.shape
    _paged_shapes(B, block_table, ctx_len)
    device = _same_device(k_pool, (v_pool, block_table, ctx_len, keep, weights, err_word))
    if k_pool.dtype == torch.uint8:
        D = head_dim
        if D is None:
            if weights is None or weights.dim() != 3 or len(pool) != 3 or weights.shape[2] == 0:
                raise ValueError("give head_dim, or weights [num_pages, Hkv, page_tokens]")
            D = max(pool[2] // weights.shape[2] - 1, 0)
        fmt, page_tokens, dtype = FP8_E4M3_PAGE, _fp8_page_tokens(k_pool, v_pool, D), BF16
    else:
        if len(pool) != 4 or v_pool.shape != pool or v_pool.dtype != k_pool.dtype:
            raise ValueError("pools must be two of [num_pages, Hkv, page_tokens, D], or FP8 pools")
        fmt, page_tokens, D, dtype = 0, pool[2], pool[3], _dt(k_pool)
        if head_dim is not None and head_dim != D:
            raise ValueError(f"the pools' rows have {D} elements")
    if keep.dim() != 3 or keep.shape[0] != B or keep.shape[1] != pool[1]:
        raise ValueError("keep must be [B, Hkv, width]")
    if weights is not None:
        _weight_pool(weights, pool[0], pool[1], page_tokens, device)
    if k_pool.shape != v_pool.shape:
        raise ValueError("k_pool and v_pool must have the same shape")
    if keep.numel() == 0:
        return
    with _launching(device, stream) as s:
        p = _COMPACT.pack(k_pool.data_ptr(), v_pool.data_ptr(), _addr(weights),
                          block_table.data_ptr(), ctx_len.data_ptr(), keep.data_ptr(),
                          _addr(err_word), dtype, fmt, B, pool[1], D, page_tokens,
                          block_table.shape[1], pool[0], keep.shape[2])
        _check("paged_kv_compact", L.paged_kv_compact_bytes(p, s))

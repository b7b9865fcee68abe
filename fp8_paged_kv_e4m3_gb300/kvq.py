"""ctypes binding of libkvq.so (include/kvq.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the cudaStream_t, and dtypes / shapes / devices are checked so
that a wrong buffer is refused before the C call.  Every step of the path
runs in the library's CUDA kernels.  There is no fallback: if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")

PAGE_SIZE = 4
KVQ_OK = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "bad scale", -3: "workspace", -4: "unsupported",
          -5: "CUDA error", -6: "alignment"}
DEV_BAD_PAGE, DEV_BAD_SLOT, DEV_BAD_TOPK, DEV_BAD_LEN, DEV_TIMEOUT, DEV_BAD_POS = 1, 2, 4, 8, 16, 32
ATTN_BITCAST_DECODE = 1
ATTN_MMA_SYNC = 2
ATTN_FP8_QK = 4
ATTN_STRICT_ORDER = 8
ATTN_LONGEST_FIRST = 32
ROPE_INTERLEAVED = 1
ROPE_SCALING = {None: 0, "linear": 1, "yarn": 2}

_lock = threading.Lock()
_lib = None
_pycall = None      # the call module, once the default library is loaded


class KvqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({status})")


class AttnParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("num_splits", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("max_topk", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("split_pages", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class PrefillParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("max_q_len", ctypes.c_int32),
                ("total_q", ctypes.c_int32), ("sm_scale", ctypes.c_float), ("flags", ctypes.c_int32)]


class RopeParams(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("max_positions", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


EXPORTS = ("kvq_version", "kvq_status_string", "kvq_validate_scales", "kvq_amax_f16",
           "kvq_scale_from_amax", "kv_append_e4m3", "kv_append_fp16", "kvq_attn_num_splits",
           "kvq_attn_workspace_bytes", "paged_decode_attn_e4m3", "paged_decode_attn_fp16",
           "paged_decode_attn_e4m3_partial", "paged_decode_attn_fp16_partial", "kvq_lse_combine",
           "paged_decode_step_e4m3", "paged_decode_step_fp16", "kvq_attn_launches",
           "paged_decode_attn_e4m3_noalloc", "kvq_prefill_workspace_bytes", "paged_prefill_attn_e4m3",
           "paged_prefill_attn_fp16", "kvq_rope_table", "kv_append_rope_e4m3", "kv_append_rope_fp16",
           "kv_append_rope_e2m1", "kvq_scale_from_amax_e2m1", "kv_append_e2m1", "kv_gather_e2m1",
           "paged_decode_attn_e2m1", "paged_decode_attn_e2m1_partial", "paged_prefill_attn_e2m1")


def load(path: Optional[str] = None):
    """Load libkvq.so (built by fp8_paged_kv_e4m3_gb300.build); raise if absent."""
    global _lib, _pycall
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library not built: {p} is missing "
                               "(run `python -m fp8_paged_kv_e4m3_gb300.build`)")
        lib = ctypes.CDLL(p)
        V, P, i32, i64, f32 = (ctypes.c_void_p, ctypes.POINTER(AttnParams), ctypes.c_int32,
                               ctypes.c_int64, ctypes.c_float)
        sz = ctypes.c_size_t
        lib.kvq_version.restype = ctypes.c_int
        lib.kvq_status_string.argtypes = [ctypes.c_int]
        lib.kvq_status_string.restype = ctypes.c_char_p
        lib.kvq_validate_scales.argtypes = [V, V, i32]
        lib.kvq_amax_f16.argtypes = [V, i64, V, V]
        lib.kvq_scale_from_amax.argtypes = [f32]
        lib.kvq_scale_from_amax.restype = f32
        lib.kv_append_e4m3.argtypes = [V, V, V, i32, i32, i32, V, V, i64, f32, f32, V, V]
        lib.kv_append_fp16.argtypes = [V, V, V, i32, i32, i32, V, V, i64, V, V]
        lib.kvq_attn_num_splits.argtypes = [P]
        lib.kvq_attn_num_splits.restype = i32
        lib.kvq_attn_launches.argtypes = [P, i32, i32]
        lib.kvq_attn_launches.restype = i32
        lib.kvq_attn_workspace_bytes.argtypes = [P]
        lib.kvq_attn_workspace_bytes.restype = sz
        lib.paged_decode_attn_e4m3.argtypes = [V, V, V, i64, V, V, f32, f32, V, V, V, sz, V, P, V, V]
        lib.paged_decode_attn_fp16.argtypes = [V, V, V, i64, V, V, V, V, V, sz, V, P, V, V]
        lib.paged_decode_attn_e4m3_partial.argtypes = [V, V, V, i64, V, V, f32, f32, V, V, V, sz, P, V, V]
        lib.paged_decode_attn_fp16_partial.argtypes = [V, V, V, i64, V, V, V, V, V, sz, P, V, V]
        lib.kvq_lse_combine.argtypes = [V, sz, V, P, V]
        lib.paged_decode_step_e4m3.argtypes = [V, V, V, V, V, i64, V, V, f32, f32, V, sz, V, P, V, V]
        lib.paged_decode_step_fp16.argtypes = [V, V, V, V, V, i64, V, V, V, sz, V, P, V, V]
        PP = ctypes.POINTER(PrefillParams)
        lib.kvq_prefill_workspace_bytes.argtypes = [PP]
        lib.kvq_prefill_workspace_bytes.restype = sz
        lib.paged_prefill_attn_e4m3.argtypes = [V, V, V, i64, V, V, V, f32, f32, V, sz, V, PP, V, V]
        lib.paged_prefill_attn_fp16.argtypes = [V, V, V, i64, V, V, V, V, sz, V, PP, V, V]
        PR, f64 = ctypes.POINTER(RopeParams), ctypes.c_double
        lib.kvq_scale_from_amax_e2m1.argtypes = [f32]
        lib.kvq_scale_from_amax_e2m1.restype = f32
        lib.kvq_rope_table.argtypes = [V, i32, i32, f64, i32, f64, i32, f64, f64, f64, V]
        lib.kv_append_rope_e4m3.argtypes = [V, V, V, V, V, V, V, V, V, i64, f32, f32, PR, V, V]
        lib.kv_append_rope_fp16.argtypes = [V, V, V, V, V, V, V, V, V, i64, PR, V, V]
        lib.kv_append_rope_e2m1.argtypes = lib.kv_append_rope_e4m3.argtypes
        lib.kv_append_e2m1.argtypes = lib.kv_append_e4m3.argtypes
        lib.kv_gather_e2m1.argtypes = [V, V, i64, V, i32, i32, i32, f32, f32, V, V, V, V]
        lib.paged_decode_attn_e2m1.argtypes = lib.paged_decode_attn_e4m3.argtypes
        lib.paged_decode_attn_e2m1_partial.argtypes = lib.paged_decode_attn_e4m3_partial.argtypes
        lib.paged_prefill_attn_e2m1.argtypes = lib.paged_prefill_attn_e4m3.argtypes
        for name in ("kvq_validate_scales", "kvq_amax_f16", "kv_append_e4m3", "kv_append_fp16",
                     "paged_decode_attn_e4m3", "paged_decode_attn_fp16",
                     "paged_decode_attn_e4m3_partial", "paged_decode_attn_fp16_partial",
                     "kvq_lse_combine", "paged_decode_step_e4m3", "paged_decode_step_fp16",
                     "paged_prefill_attn_e4m3", "paged_prefill_attn_fp16", "kvq_rope_table",
                     "kv_append_rope_e4m3", "kv_append_rope_fp16", "kv_append_rope_e2m1", "kv_append_e2m1",
                     "kv_gather_e2m1", "paged_decode_attn_e2m1", "paged_decode_attn_e2m1_partial",
                     "paged_prefill_attn_e2m1"):
            getattr(lib, name).restype = ctypes.c_int
        if path is None:
            _pycall = _load_pycall(lib, os.path.join(os.path.dirname(p), "kvq_pycall.so"))
            _lib = lib
        return lib


def _load_pycall(lib, path: str):
    """The CPython module that marshals the E2M1 and rotary calls (kvq_pycall.cpp).  Its functions return a
    status, or None for arguments that are not those of a plain call: the ctypes path then names them."""
    if not os.path.exists(path):
        raise RuntimeError(f"call module not built: {path} is missing (run `python -m fp8_paged_kv_e4m3_gb300.build`)")
    spec = importlib.util.spec_from_file_location("kvq_pycall", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    entry = ("paged_decode_attn_e2m1", "paged_decode_attn_e2m1_partial", "paged_prefill_attn_e2m1", "kv_append_e2m1",
             "kv_gather_e2m1", "kv_append_rope_e4m3", "kv_append_rope_e2m1", "kv_append_rope_fp16")
    mod.setup(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in entry),
              _raw_stream, getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
    return mod


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):   # the same value, without a Python stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream


def _check(fn: str, status: int):
    if status != KVQ_OK:
        raise KvqError(fn, status)


# ---------------------------------------------------------------------------
# marshalling helpers

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, ndim: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {tuple(t.shape)}")


# ---------------------------------------------------------------------------
# scales and calibration

def validate_scales(k_scales, v_scales) -> None:
    """Fail closed unless every per-layer K and V scale is finite and > 0."""
    k = (ctypes.c_float * len(k_scales))(*[float(x) for x in k_scales])
    v = (ctypes.c_float * len(v_scales))(*[float(x) for x in v_scales])
    if len(k_scales) != len(v_scales) or len(k_scales) == 0:
        raise KvqError("kvq_validate_scales", -1)
    _check("kvq_validate_scales", load().kvq_validate_scales(k, v, len(k_scales)))


def amax_f16(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """max |x| over an fp16 device tensor, as a device float32[1] (no host sync)."""
    _need(x, "x", torch.float16)
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _need(out, "amax_out", torch.float32)
    _check("kvq_amax_f16", load().kvq_amax_f16(_ptr(x), x.numel(), _ptr(out), _stream(x)))
    return out


def scale_from_amax(amax: float) -> float:
    return float(load().kvq_scale_from_amax(ctypes.c_float(amax)))


def calibrate_scale(x: torch.Tensor) -> float:
    """scale = amax / 448 of a calibration draw (synchronises to read amax)."""
    return scale_from_amax(float(amax_f16(x).item()))


# ---------------------------------------------------------------------------
# append

def _append_common(k_new, v_new, slot_mapping, k_cache, v_cache, cache_dtype):
    _need(k_new, "k_new", torch.float16, 3)
    _need(v_new, "v_new", torch.float16, 3)
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new shapes differ")
    T, Hkv, D = k_new.shape
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping length != number of tokens")
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(c, name, cache_dtype, 4)
        if c.shape[1:] != (Hkv, PAGE_SIZE, D):
            raise ValueError(f"{name}: expected [P, {Hkv}, {PAGE_SIZE}, {D}], got {tuple(c.shape)}")
    return T, Hkv, D


def kv_append_e4m3(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale: float, v_scale: float,
                   err_flag: Optional[torch.Tensor] = None) -> None:
    """Quantise fp16 K/V of new tokens into uint8 (E4M3) pools [P][Hkv][4][D]."""
    T, Hkv, D = _append_common(k_new, v_new, slot_mapping, k_cache, v_cache, torch.uint8)
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    _check("kv_append_e4m3", load().kv_append_e4m3(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T, Hkv, D, _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(err_flag),
        _stream(k_new)))


def kv_append_fp16(k_new, v_new, slot_mapping, k_cache, v_cache,
                   err_flag: Optional[torch.Tensor] = None) -> None:
    T, Hkv, D = _append_common(k_new, v_new, slot_mapping, k_cache, v_cache, torch.float16)
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    _check("kv_append_fp16", load().kv_append_fp16(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T, Hkv, D, _ptr(k_cache), _ptr(v_cache),
        k_cache.shape[0], _ptr(err_flag), _stream(k_new)))


# ---------------------------------------------------------------------------
# attention

def attn_params(q: torch.Tensor, num_kv_heads: int, max_pages_per_seq: int, num_splits: int = 0,
                max_topk: int = 0, sm_scale: float = 0.0, split_pages: int = 0,
                bitcast_decode: bool = False, mma_sync: bool = False, fp8_qk: bool = False,
                strict_order: bool = False, longest_first: bool = False) -> AttnParams:
    B, q_len, Hq, D = q.shape
    return AttnParams(B, q_len, Hq, num_kv_heads, D, num_splits, max_pages_per_seq, max_topk,
                      sm_scale, split_pages,
                      _flags(bitcast_decode, mma_sync, fp8_qk, strict_order, longest_first))


def _flags(bitcast_decode: bool, mma_sync: bool, fp8_qk: bool = False, strict_order: bool = False,
           longest_first: bool = False) -> int:
    return ((ATTN_BITCAST_DECODE if bitcast_decode else 0) | (ATTN_MMA_SYNC if mma_sync else 0) |
            (ATTN_FP8_QK if fp8_qk else 0) | (ATTN_STRICT_ORDER if strict_order else 0) |
            (ATTN_LONGEST_FIRST if longest_first else 0))


def num_splits(p: AttnParams) -> int:
    s = load().kvq_attn_num_splits(ctypes.byref(p))
    if s < 1:
        raise KvqError("kvq_attn_num_splits", s)
    return s


def attn_launches(p: AttnParams, e4m3: bool, fused_step: bool = False) -> int:
    """Kernels the full call (fused_step: the fused step call) launches with
    these parameters on the current device."""
    n = load().kvq_attn_launches(ctypes.byref(p), int(e4m3), int(fused_step))
    if n < 0:
        raise KvqError("kvq_attn_launches", n)
    return n


def workspace_bytes(p: AttnParams) -> int:
    n = load().kvq_attn_workspace_bytes(ctypes.byref(p))
    if n == 0:
        raise KvqError("kvq_attn_workspace_bytes", -1)
    return n


def alloc_workspace(p: AttnParams, device) -> torch.Tensor:
    """An FP32 workspace of the size the call needs (caller-owned)."""
    return torch.empty(math.ceil(workspace_bytes(p) / 4), dtype=torch.float32, device=device)


def workspace_views(ws: torch.Tensor, p: AttnParams):
    """(tmp_out [B][Hq][q_len][S][D], tmp_max [B][Hq][q_len][S], tmp_sum) views of a workspace."""
    S = num_splits(p)
    units = p.batch * p.num_q_heads * p.q_len * S
    r256 = lambda n: (n + 255) // 256 * 256
    o_n = units * p.head_dim
    m_off = r256(o_n * 4) // 4
    l_off = m_off + r256(units * 4) // 4
    shp = (p.batch, p.num_q_heads, p.q_len, S)
    return (ws[:o_n].view(*shp, p.head_dim), ws[m_off:m_off + units].view(shp),
            ws[l_off:l_off + units].view(shp))


def e2m1_page_bytes(head_dim: int) -> int:
    """Bytes of one E2M1 page of one kv head: 4 tokens' codes and block scales."""
    return 9 * head_dim // 4


def _pools(k_cache, v_cache, dtype, D: int, e2m1: bool = False) -> int:
    """Check a K and a V pool of head_dim D; returns the kv heads."""
    tail = (e2m1_page_bytes(D),) if e2m1 else (PAGE_SIZE, D)
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(c, name, dtype, 2 + len(tail))
        if c.shape != k_cache.shape or tuple(c.shape[2:]) != tail:
            raise ValueError(f"caches must be [P, Hkv, {', '.join(map(str, tail))}]")
    return k_cache.shape[1]


def _same_device(like: torch.Tensor, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != like.device:
            raise ValueError(f"{name}: on {t.device}, expected {like.device}")


def _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, out, topk_idx,
                topk_lens, cache_dtype, num_splits_, sm_scale, split_pages, bitcast_decode=False,
                mma_sync=False, fp8_qk=False, strict_order=False, longest_first=False, e2m1=False):
    _need(q, "q", torch.float16, 4)
    B, q_len, Hq, D = q.shape
    Hkv = _pools(k_cache, v_cache, cache_dtype, D, e2m1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch mismatch")
    # the split workspace is FP32 by contract; an fp16 buffer is refused here
    _need(workspace, "workspace", torch.float32)
    if out is not None:
        _need(out, "out", torch.float16, 4)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    max_topk = 0
    if (topk_idx is None) != (topk_lens is None):
        raise ValueError("topk_idx and topk_lens go together")
    if topk_idx is not None:
        _need(topk_idx, "topk_idx", torch.int32, 3)
        _need(topk_lens, "topk_lens", torch.int32, 1)
        if topk_idx.shape[:2] != (B, Hkv) or topk_lens.shape[0] != B:
            raise ValueError("topk_idx must be [B, Hkv, K], topk_lens [B]")
        max_topk = topk_idx.shape[2]
    p = AttnParams(B, q_len, Hq, Hkv, D, num_splits_, block_tables.shape[1], max_topk, sm_scale,
                   split_pages, _flags(bitcast_decode, mma_sync, fp8_qk, strict_order, longest_first))
    return p


def paged_decode_attn_e4m3(q, k_cache, v_cache, block_tables, context_lens, k_scale: float,
                           v_scale: float, workspace, out=None, topk_idx=None, topk_lens=None,
                           num_splits: int = 0, sm_scale: float = 0.0, err_flag=None,
                           split_pages: int = 0, bitcast_decode: bool = False, mma_sync: bool = False,
                           fp8_qk: bool = False, strict_order: bool = False, longest_first: bool = False):
    """Decode / verify attention over E4M3 pools; returns `out` (fp16, shape of q).
    fp8_qk: scores from the query quantised to E4M3 per (sequence, kv head)
    on E4M3 tensor-core instructions (verify shapes at head_dim 128 only).
    strict_order: read no input before the preceding kernel in the stream
    completes (by default, without a top-k list, block tables, lengths and
    the pages of positions below L - q_len may be read earlier).
    longest_first: the split kernel takes the sequences longest first (for
    batches of varied lengths over several waves; same results)."""
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, out, topk_idx,
                    topk_lens, torch.uint8, num_splits, sm_scale, split_pages, bitcast_decode, mma_sync,
                    fp8_qk, strict_order, longest_first)
    if out is None:
        out = torch.empty_like(q)
    _check("paged_decode_attn_e4m3", load().paged_decode_attn_e4m3(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables),
        _ptr(context_lens), ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(topk_idx),
        _ptr(topk_lens), _ptr(workspace), workspace.numel() * 4, _ptr(out), ctypes.byref(p),
        _ptr(err_flag), _stream(q)))
    return out


def paged_decode_attn_fp16(q, k_cache, v_cache, block_tables, context_lens, workspace, out=None,
                           topk_idx=None, topk_lens=None, num_splits: int = 0,
                           sm_scale: float = 0.0, err_flag=None, split_pages: int = 0,
                           mma_sync: bool = False, strict_order: bool = False, longest_first: bool = False):
    """fp16-KV twin of paged_decode_attn_e4m3."""
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, out, topk_idx,
                    topk_lens, torch.float16, num_splits, sm_scale, split_pages, False, mma_sync,
                    strict_order=strict_order, longest_first=longest_first)
    if out is None:
        out = torch.empty_like(q)
    _check("paged_decode_attn_fp16", load().paged_decode_attn_fp16(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables),
        _ptr(context_lens), _ptr(topk_idx), _ptr(topk_lens), _ptr(workspace),
        workspace.numel() * 4, _ptr(out), ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return out


def _step_rows_check(q, k_new, v_new, Hkv):
    B, q_len, _, D = q.shape
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _need(t, name, torch.float16, 4)
        if t.shape != (B, q_len, Hkv, D):
            raise ValueError(f"{name} must be [B, q_len, Hkv, D] = {(B, q_len, Hkv, D)}")


def paged_decode_step_e4m3(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, k_scale: float,
                           v_scale: float, workspace, out=None, num_splits: int = 0, sm_scale: float = 0.0,
                           err_flag=None, split_pages: int = 0, bitcast_decode: bool = False,
                           mma_sync: bool = False, fp8_qk: bool = False, strict_order: bool = False,
                           longest_first: bool = False):
    """This step's append (k_new, v_new: fp16 [B, q_len, Hkv, D], written at
    positions L - q_len .. L - 1 of each sequence) and the attention over the
    updated cache in one attention launch plus the combine; the same pools
    and outputs as kv_append_e4m3 then paged_decode_attn_e4m3.  Returns out."""
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, out, None, None,
                    torch.uint8, num_splits, sm_scale, split_pages, bitcast_decode, mma_sync, fp8_qk,
                    strict_order, longest_first)
    _step_rows_check(q, k_new, v_new, k_cache.shape[1])
    if out is None:
        out = torch.empty_like(q)
    _check("paged_decode_step_e4m3", load().paged_decode_step_e4m3(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(block_tables), _ptr(context_lens), ctypes.c_float(k_scale), ctypes.c_float(v_scale),
        _ptr(workspace), workspace.numel() * 4, _ptr(out), ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return out


def paged_decode_step_fp16(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, workspace,
                           out=None, num_splits: int = 0, sm_scale: float = 0.0, err_flag=None,
                           split_pages: int = 0, mma_sync: bool = False, strict_order: bool = False,
                           longest_first: bool = False):
    """fp16-KV twin of paged_decode_step_e4m3."""
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, out, None, None,
                    torch.float16, num_splits, sm_scale, split_pages, False, mma_sync,
                    strict_order=strict_order, longest_first=longest_first)
    _step_rows_check(q, k_new, v_new, k_cache.shape[1])
    if out is None:
        out = torch.empty_like(q)
    _check("paged_decode_step_fp16", load().paged_decode_step_fp16(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(block_tables), _ptr(context_lens), _ptr(workspace), workspace.numel() * 4, _ptr(out),
        ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return out


def paged_decode_attn_e4m3_partial(q, k_cache, v_cache, block_tables, context_lens,
                                   k_scale: float, v_scale: float, workspace, topk_idx=None,
                                   topk_lens=None, num_splits: int = 0, sm_scale: float = 0.0,
                                   err_flag=None, split_pages: int = 0,
                                   bitcast_decode: bool = False, mma_sync: bool = False,
                                   fp8_qk: bool = False, strict_order: bool = False,
                                   longest_first: bool = False) -> AttnParams:
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, None, topk_idx,
                    topk_lens, torch.uint8, num_splits, sm_scale, split_pages, bitcast_decode, mma_sync,
                    fp8_qk, strict_order, longest_first)
    _check("paged_decode_attn_e4m3_partial", load().paged_decode_attn_e4m3_partial(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables),
        _ptr(context_lens), ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(topk_idx),
        _ptr(topk_lens), _ptr(workspace), workspace.numel() * 4, ctypes.byref(p),
        _ptr(err_flag), _stream(q)))
    return p


def paged_decode_attn_fp16_partial(q, k_cache, v_cache, block_tables, context_lens, workspace,
                                   topk_idx=None, topk_lens=None, num_splits: int = 0,
                                   sm_scale: float = 0.0, err_flag=None,
                                   split_pages: int = 0, mma_sync: bool = False,
                                   strict_order: bool = False, longest_first: bool = False) -> AttnParams:
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, None, topk_idx,
                    topk_lens, torch.float16, num_splits, sm_scale, split_pages, False, mma_sync,
                    strict_order=strict_order, longest_first=longest_first)
    _check("paged_decode_attn_fp16_partial", load().paged_decode_attn_fp16_partial(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables),
        _ptr(context_lens), _ptr(topk_idx), _ptr(topk_lens), _ptr(workspace),
        workspace.numel() * 4, ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return p


def lse_combine(workspace: torch.Tensor, out: torch.Tensor, p: AttnParams) -> torch.Tensor:
    _need(workspace, "workspace", torch.float32)
    _need(out, "out", torch.float16, 4)
    _check("kvq_lse_combine", load().kvq_lse_combine(
        _ptr(workspace), workspace.numel() * 4, _ptr(out), ctypes.byref(p), _stream(out)))
    return out


# ---------------------------------------------------------------------------
# chunked prefill

def prefill_params(q: torch.Tensor, num_kv_heads: int, batch: int, max_pages_per_seq: int,
                   max_q_len: int, sm_scale: float = 0.0) -> PrefillParams:
    """Parameters of a prefill call; q is the packed [total_q, Hq, D] chunk tensor."""
    return PrefillParams(batch, q.shape[1], num_kv_heads, q.shape[2], max_pages_per_seq, max_q_len,
                         q.shape[0], sm_scale, 0)


def prefill_workspace_bytes(p: PrefillParams) -> int:
    n = int(load().kvq_prefill_workspace_bytes(ctypes.byref(p)))
    if n == 0:
        raise KvqError("kvq_prefill_workspace_bytes", -1)
    return n


def alloc_prefill_workspace(p: PrefillParams, device) -> torch.Tensor:
    return torch.empty(prefill_workspace_bytes(p), dtype=torch.uint8, device=device)


def _prefill_check(q, k_cache, v_cache, block_tables, context_lens, q_start, workspace, out,
                   cache_dtype, max_q_len, sm_scale, e2m1=False):
    _need(q, "q", torch.float16, 3)
    Tq, Hq, D = q.shape
    _pools(k_cache, v_cache, cache_dtype, D, e2m1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(q_start, "q_start", torch.int32, 1)
    B = context_lens.shape[0]
    if block_tables.shape[0] != B or q_start.shape[0] != B + 1:
        raise ValueError("block_tables [B, max_pages], context_lens [B], q_start [B + 1] expected")
    _need(workspace, "workspace", torch.uint8, 1)
    if out is not None:
        _need(out, "out", torch.float16, 3)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    if max_q_len is None:
        max_q_len = max(1, Tq)
    return PrefillParams(B, Hq, k_cache.shape[1], D, block_tables.shape[1], max_q_len, Tq, sm_scale, 0)


def paged_prefill_attn_e4m3(q, k_cache, v_cache, block_tables, context_lens, q_start, k_scale: float,
                            v_scale: float, workspace, out=None, max_q_len: Optional[int] = None,
                            sm_scale: float = 0.0, err_flag=None):
    """Chunked-prefill attention over E4M3 pools; q and the returned out are [total_q, Hq, D] fp16,
    q_start [B + 1] the chunk offsets.  max_q_len bounds every chunk (default: total_q)."""
    p = _prefill_check(q, k_cache, v_cache, block_tables, context_lens, q_start, workspace, out,
                       torch.uint8, max_q_len, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    _check("paged_prefill_attn_e4m3", load().paged_prefill_attn_e4m3(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables), _ptr(context_lens),
        _ptr(q_start), ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(workspace), workspace.numel(),
        _ptr(out), ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return out


def paged_prefill_attn_fp16(q, k_cache, v_cache, block_tables, context_lens, q_start, workspace, out=None,
                            max_q_len: Optional[int] = None, sm_scale: float = 0.0, err_flag=None):
    """fp16-KV twin of paged_prefill_attn_e4m3."""
    p = _prefill_check(q, k_cache, v_cache, block_tables, context_lens, q_start, workspace, out,
                       torch.float16, max_q_len, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    _check("paged_prefill_attn_fp16", load().paged_prefill_attn_fp16(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables), _ptr(context_lens),
        _ptr(q_start), _ptr(workspace), workspace.numel(), _ptr(out), ctypes.byref(p), _ptr(err_flag),
        _stream(q)))
    return out


# ---------------------------------------------------------------------------
# rotary positions, and the append with the rotation on the way

def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original_positions: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
               magnitude: float = 0.0, device="cuda") -> torch.Tensor:
    """The float32 [max_positions, rot_dim] table (cos, then sin, of every
    position's angles) that the kv_append_rope_* calls read.  scaling: None,
    "linear" (factor) or "yarn" (factor, original_positions, beta_fast,
    beta_slow); magnitude 0 = 1, or 0.1 ln(factor) + 1 with "yarn"."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling: expected one of {list(ROPE_SCALING)}")
    if max_positions < 1 or rot_dim < 1 or rot_dim % 16:
        raise ValueError("max_positions and rot_dim must be positive, rot_dim a multiple of 16")
    table = torch.empty(max_positions, rot_dim, dtype=torch.float32, device=device)
    with torch.cuda.device(table.device):
        _check("kvq_rope_table", load().kvq_rope_table(
            _ptr(table), max_positions, rot_dim, base, ROPE_SCALING[scaling], factor, original_positions, beta_fast,
            beta_slow, magnitude, _stream(table)))
    return table


def _heads(t, name: str):
    """An fp16 [T, H, D] CUDA tensor whose heads are contiguous; any token stride (a slice of a packed
    projection).  Returns the stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != torch.float16:
        raise TypeError(f"{name}: expected {torch.float16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected 3 dims, got {tuple(t.shape)}")
    T, H, D = t.shape
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if T <= 1:
        return H * D
    if t.stride(0) < H * D:
        raise ValueError(f"{name}: tokens overlap")
    return t.stride(0)


def _append_rope(fn, q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache, scales, dtype, e2m1, q_out,
                 interleaved, err_flag):
    ks, vs = _heads(k_new, "k_new"), _heads(v_new, "v_new")
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new shapes differ")
    T, Hkv, D = k_new.shape
    Hq = qs = 0
    if q is not None:
        qs = _heads(q, "q")
        Hq = q.shape[1]
        if q.shape[0] != T or q.shape[2] != D or Hq < 1:
            raise ValueError(f"q must be [{T}, Hq, {D}], got {tuple(q.shape)}")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _need(q_out, "q_out", torch.float16, 3)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
    elif q_out is not None:
        raise ValueError("q_out without q")
    _need(positions, "positions", torch.int32, 1)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    if positions.numel() != T or slot_mapping.numel() != T:
        raise ValueError("positions / slot_mapping length != number of tokens")
    _need(table, "table", torch.float32, 2)
    if _pools(k_cache, v_cache, dtype, D, e2m1) != Hkv:
        raise ValueError(f"the pools hold {k_cache.shape[1]} kv heads, k_new has {Hkv}")
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    _same_device(k_new, q=q, q_out=q_out, v_new=v_new, positions=positions, table=table, slot_mapping=slot_mapping,
                 k_cache=k_cache, v_cache=v_cache, err_flag=err_flag)
    p = RopeParams(T, Hq, Hkv, D, table.shape[1], table.shape[0], ROPE_INTERLEAVED if interleaved else 0, qs, ks, vs)
    with torch.cuda.device(k_new.device):
        _check(fn, getattr(load(), fn)(
            _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(table), _ptr(slot_mapping), _ptr(q_out),
            _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], *[ctypes.c_float(s) for s in scales], ctypes.byref(p),
            _ptr(err_flag), _stream(k_new)))
    return q_out


def kv_append_rope_e4m3(q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache, k_scale: float, v_scale: float,
                        q_out=None, interleaved: bool = False, err_flag: Optional[torch.Tensor] = None):
    """Rotate q [T, Hq, D] (None: no queries) and k_new [T, Hkv, D] by their
    positions and append K and V to uint8 (E4M3) pools, in one launch.
    table: rope_table(...), whose width is the rotated part of the head.
    interleaved: pairs (2j, 2j + 1) instead of (j, j + rot_dim / 2).  q, k_new
    and v_new may be slices of one packed projection; q_out may be q itself
    when that is contiguous.  Returns q_out."""
    if _pycall is not None:
        if q_out is None and q is not None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        st = _pycall.rope(0, q, k_new, v_new, positions, table, slot_mapping, q_out, k_cache, v_cache, k_scale, v_scale,
                          ROPE_INTERLEAVED if interleaved else 0, err_flag)
        if st == KVQ_OK:
            return q_out
        if st is not None:
            raise KvqError("kv_append_rope_e4m3", st)
    return _append_rope("kv_append_rope_e4m3", q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache,
                        (k_scale, v_scale), torch.uint8, False, q_out, interleaved, err_flag)


def kv_append_rope_fp16(q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache, q_out=None,
                        interleaved: bool = False, err_flag: Optional[torch.Tensor] = None):
    """fp16-KV twin of kv_append_rope_e4m3."""
    if _pycall is not None:
        if q_out is None and q is not None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        st = _pycall.rope(1, q, k_new, v_new, positions, table, slot_mapping, q_out, k_cache, v_cache, 1.0, 1.0,
                          ROPE_INTERLEAVED if interleaved else 0, err_flag)
        if st == KVQ_OK:
            return q_out
        if st is not None:
            raise KvqError("kv_append_rope_fp16", st)
    return _append_rope("kv_append_rope_fp16", q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache, (),
                        torch.float16, False, q_out, interleaved, err_flag)


def kv_append_rope_e2m1(q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache, k_scale: float, v_scale: float,
                        q_out=None, interleaved: bool = False, err_flag: Optional[torch.Tensor] = None):
    """kv_append_rope_e4m3 into E2M1 pools."""
    if _pycall is not None:
        if q_out is None and q is not None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        st = _pycall.rope(2, q, k_new, v_new, positions, table, slot_mapping, q_out, k_cache, v_cache, k_scale, v_scale,
                          ROPE_INTERLEAVED if interleaved else 0, err_flag)
        if st == KVQ_OK:
            return q_out
        if st is not None:
            raise KvqError("kv_append_rope_e2m1", st)
    return _append_rope("kv_append_rope_e2m1", q, k_new, v_new, positions, table, slot_mapping, k_cache, v_cache,
                        (k_scale, v_scale), torch.uint8, True, q_out, interleaved, err_flag)


# ---------------------------------------------------------------------------
# the 4-bit cache

def scale_from_amax_e2m1(amax: float) -> float:
    return float(load().kvq_scale_from_amax_e2m1(ctypes.c_float(amax)))


def calibrate_scale_e2m1(x: torch.Tensor) -> float:
    """scale = amax / 2688 of a calibration draw (synchronises to read amax)."""
    return scale_from_amax_e2m1(float(amax_f16(x).item()))


def alloc_e2m1_pool(num_pages: int, num_kv_heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """A zeroed E2M1 pool, uint8 [num_pages, num_kv_heads, 9 * head_dim / 4]."""
    return torch.zeros(num_pages, num_kv_heads, e2m1_page_bytes(head_dim), dtype=torch.uint8, device=device)


def kv_append_e2m1(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale: float, v_scale: float,
                   err_flag: Optional[torch.Tensor] = None) -> None:
    """Quantise fp16 K/V of new tokens [T, Hkv, D] into E2M1 pools."""
    if _pycall is not None:
        st = _pycall.append(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, err_flag)
        if st is not None:
            return _check("kv_append_e2m1", st)
    _need(k_new, "k_new", torch.float16, 3)
    _need(v_new, "v_new", torch.float16, 3)
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new shapes differ")
    T, Hkv, D = k_new.shape
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping length != number of tokens")
    if _pools(k_cache, v_cache, torch.uint8, D, True) != Hkv:
        raise ValueError(f"the pools hold {k_cache.shape[1]} kv heads, k_new has {Hkv}")
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    _same_device(k_new, v_new=v_new, slot_mapping=slot_mapping, k_cache=k_cache, v_cache=v_cache, err_flag=err_flag)
    with torch.cuda.device(k_new.device):
        _check("kv_append_e2m1", load().kv_append_e2m1(
            _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T, Hkv, D, _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
            ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(err_flag), _stream(k_new)))


def kv_gather_e2m1(k_cache, v_cache, slots, k_scale: float, v_scale: float, k_out=None, v_out=None,
                   err_flag: Optional[torch.Tensor] = None):
    """The cached rows at `slots` as fp16 [T, Hkv, D] (K, V); zeros for a slot of -1."""
    if _pycall is not None and k_out is not None and v_out is not None:
        st = _pycall.gather(k_cache, v_cache, slots, k_scale, v_scale, k_out, v_out, err_flag)
        if st is not None:
            _check("kv_gather_e2m1", st)
            return k_out, v_out
    _need(k_cache, "k_cache", torch.uint8, 3)
    D = k_cache.shape[2] * 4 // 9
    Hkv = _pools(k_cache, v_cache, torch.uint8, D, True)
    _need(slots, "slots", torch.int32, 1)
    shape = (slots.numel(), Hkv, D)
    k_out, v_out = (torch.empty(shape, dtype=torch.float16, device=k_cache.device) if t is None else t
                    for t in (k_out, v_out))
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _need(t, name, torch.float16, 3)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name}: expected {shape}, got {tuple(t.shape)}")
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32)
    _same_device(k_cache, v_cache=v_cache, slots=slots, k_out=k_out, v_out=v_out, err_flag=err_flag)
    with torch.cuda.device(k_cache.device):
        _check("kv_gather_e2m1", load().kv_gather_e2m1(
            _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(slots), slots.numel(), Hkv, D, ctypes.c_float(k_scale),
            ctypes.c_float(v_scale), _ptr(k_out), _ptr(v_out), _ptr(err_flag), _stream(k_cache)))
    return k_out, v_out


def _e2m1_devices(q, **tensors):
    if tensors.get("err_flag") is not None:
        _need(tensors["err_flag"], "err_flag", torch.int32)
    _same_device(q, **tensors)


def paged_decode_attn_e2m1(q, k_cache, v_cache, block_tables, context_lens, k_scale: float, v_scale: float, workspace,
                           out=None, topk_idx=None, topk_lens=None, num_splits: int = 0, sm_scale: float = 0.0,
                           err_flag=None, split_pages: int = 0, strict_order: bool = False):
    """paged_decode_attn_e4m3 over E2M1 pools [P, Hkv, 9 * D / 4]; returns `out` (fp16, shape of q)."""
    if _pycall is not None:
        if out is None:
            out = torch.empty_like(q)
        st = _pycall.decode(q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, workspace, out, topk_idx,
                            topk_lens, num_splits, sm_scale, err_flag, split_pages, ATTN_STRICT_ORDER if strict_order else 0)
        if st is not None:
            _check("paged_decode_attn_e2m1", st)
            return out
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, out, topk_idx, topk_lens, torch.uint8,
                    num_splits, sm_scale, split_pages, strict_order=strict_order, e2m1=True)
    _e2m1_devices(q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables, context_lens=context_lens,
                  workspace=workspace, out=out, topk_idx=topk_idx, topk_lens=topk_lens, err_flag=err_flag)
    if out is None:
        out = torch.empty_like(q)
    with torch.cuda.device(q.device):
        _check("paged_decode_attn_e2m1", load().paged_decode_attn_e2m1(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables), _ptr(context_lens),
            ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(topk_idx), _ptr(topk_lens), _ptr(workspace),
            workspace.numel() * 4, _ptr(out), ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return out


def paged_decode_attn_e2m1_partial(q, k_cache, v_cache, block_tables, context_lens, k_scale: float, v_scale: float,
                                   workspace, topk_idx=None, topk_lens=None, num_splits: int = 0, sm_scale: float = 0.0,
                                   err_flag=None, split_pages: int = 0, strict_order: bool = False) -> AttnParams:
    p = _attn_check(q, k_cache, v_cache, block_tables, context_lens, workspace, None, topk_idx, topk_lens, torch.uint8,
                    num_splits, sm_scale, split_pages, strict_order=strict_order, e2m1=True)
    _e2m1_devices(q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables, context_lens=context_lens,
                  workspace=workspace, topk_idx=topk_idx, topk_lens=topk_lens, err_flag=err_flag)
    with torch.cuda.device(q.device):
        _check("paged_decode_attn_e2m1_partial", load().paged_decode_attn_e2m1_partial(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables), _ptr(context_lens),
            ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(topk_idx), _ptr(topk_lens), _ptr(workspace),
            workspace.numel() * 4, ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return p


def paged_prefill_attn_e2m1(q, k_cache, v_cache, block_tables, context_lens, q_start, k_scale: float, v_scale: float,
                            workspace, out=None, max_q_len: Optional[int] = None, sm_scale: float = 0.0, err_flag=None):
    """paged_prefill_attn_e4m3 over E2M1 pools [P, Hkv, 288]."""
    if _pycall is not None and max_q_len is not None:
        if out is None:
            out = torch.empty_like(q)
        st = _pycall.prefill(q, k_cache, v_cache, block_tables, context_lens, q_start, k_scale, v_scale, workspace, out,
                             max_q_len, sm_scale, err_flag)
        if st is not None:
            _check("paged_prefill_attn_e2m1", st)
            return out
    p = _prefill_check(q, k_cache, v_cache, block_tables, context_lens, q_start, workspace, out, torch.uint8, max_q_len,
                       sm_scale, e2m1=True)
    _e2m1_devices(q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables, context_lens=context_lens,
                  q_start=q_start, workspace=workspace, out=out, err_flag=err_flag)
    if out is None:
        out = torch.empty_like(q)
    with torch.cuda.device(q.device):
        _check("paged_prefill_attn_e2m1", load().paged_prefill_attn_e2m1(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(block_tables), _ptr(context_lens),
            _ptr(q_start), ctypes.c_float(k_scale), ctypes.c_float(v_scale), _ptr(workspace), workspace.numel(),
            _ptr(out), ctypes.byref(p), _ptr(err_flag), _stream(q)))
    return out

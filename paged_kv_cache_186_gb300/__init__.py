"""Python binding of the sm_103a paged-KV-cache attention library.

Thin ctypes marshalling over the C ABI declared in include/pa.h: tensors are
passed as device pointers, the stream is torch's current CUDA stream. Every
step of the computation runs in the library's CUDA kernels; this module never
computes attention itself and has no fallback. If libpa_gb300.so is missing,
every call raises (build it with ``python -m paged_kv_cache_186_gb300.build``).

Names follow the C ABI: store_kv, decode, decode_window, decode_append,
decode_workspace_size, prefill_varlen, decode_noalloc, get_device_error,
debug_inject_wait_timeout; for a decode loop over a bounded cache:
norm_rope_store, prefill_window, decode_scored, decode_scored_workspace_size,
evict; for many requests over one shared context: norm_rope_axes_store,
decode_shared, decode_shared_workspace_size, prefill_shared,
prefill_shared_workspace_size.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa_gb300.so")

PA_KV_BF16 = 0
PA_KV_FP8_E4M3 = 1
PA_KV_INT8 = 2

PA_DEVERR_SLOT_RANGE = 0x1
PA_DEVERR_WAIT_TIMEOUT = 0x2
PA_DEVERR_BLOCK_RANGE = 0x4
PA_DEVERR_POSITION_RANGE = 0x8

STATUS = {0: "PA_OK", 1: "PA_ERR_NULL", 2: "PA_ERR_SHAPE", 3: "PA_ERR_DTYPE",
          4: "PA_ERR_UNSUPPORTED", 5: "PA_ERR_CUDA", 6: "PA_ERR_WORKSPACE", 7: "PA_ERR_ALIGN",
          8: "PA_ERR_TOO_LARGE"}

# Size of the static scratch buffer pa_decode_noalloc uses (PA_DECODE_NOALLOC_SCRATCH_BYTES).
DECODE_NOALLOC_SCRATCH_BYTES = 32 << 20

# Every symbol include/pa.h declares.
EXPORTED = ("pa_abi_version", "pa_status_string", "pa_store_kv", "pa_decode_workspace_size",
            "pa_decode", "pa_decode_window", "pa_decode_append", "pa_decode_window_append",
            "pa_prefill_varlen", "pa_norm_rope_store", "pa_prefill_window", "pa_decode_scored",
            "pa_decode_scored_workspace_size", "pa_evict", "pa_norm_rope_axes_store",
            "pa_decode_shared", "pa_decode_shared_workspace_size", "pa_prefill_shared",
            "pa_prefill_shared_workspace_size",
            "pa_decode_noalloc", "pa_get_device_error", "pa_debug_inject_wait_timeout")


class PAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


class KVCache(ctypes.Structure):
    """Mirror of pa_kv_cache."""
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class NormRope(ctypes.Structure):
    """Mirror of pa_norm_rope."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("cos_sin", ctypes.c_void_p), ("max_positions", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libpa_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m paged_kv_cache_186_gb300.build` (needs nvcc)")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.pa_abi_version.restype = i32
    L.pa_abi_version.argtypes = []
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_status_string.argtypes = [ctypes.c_int]
    L.pa_store_kv.restype = ctypes.c_int
    L.pa_store_kv.argtypes = [P, P, P, P, P, i32, ctypes.POINTER(KVCache), P]
    L.pa_decode_workspace_size.restype = ctypes.c_size_t
    L.pa_decode_workspace_size.argtypes = [ctypes.POINTER(KVCache), i32, i32, i32, i32]
    L.pa_decode.restype = ctypes.c_int
    L.pa_decode.argtypes = [P, ctypes.POINTER(KVCache), P, i32, P, i32, i32, i32, ctypes.c_float,
                            P, P, ctypes.c_size_t, P]
    L.pa_decode_window.restype = ctypes.c_int
    L.pa_decode_window.argtypes = [P, ctypes.POINTER(KVCache), P, i32, P, i32, i32, i32,
                                   ctypes.c_float, i32, i32, P, P, ctypes.c_size_t, P]
    L.pa_decode_append.restype = ctypes.c_int
    L.pa_decode_append.argtypes = [P, P, P, P, P, ctypes.POINTER(KVCache), P, i32, P, i32, i32,
                                   i32, ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.pa_decode_window_append.restype = ctypes.c_int
    L.pa_decode_window_append.argtypes = [P, P, P, P, P, ctypes.POINTER(KVCache), P, i32, P, i32,
                                          i32, i32, ctypes.c_float, i32, i32, P, P,
                                          ctypes.c_size_t, P]
    L.pa_prefill_varlen.restype = ctypes.c_int
    L.pa_prefill_varlen.argtypes = [P, ctypes.POINTER(KVCache), P, i32, P, P, i32, i32, i32, i32,
                                    ctypes.c_float, P, P]
    L.pa_decode_noalloc.restype = ctypes.c_int
    L.pa_decode_noalloc.argtypes = [P, ctypes.POINTER(KVCache), P, i32, P, i32, i32, i32,
                                    ctypes.c_float, P, P]
    L.pa_get_device_error.restype = ctypes.c_int
    L.pa_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.pa_debug_inject_wait_timeout.restype = ctypes.c_int
    L.pa_debug_inject_wait_timeout.argtypes = [i32, ctypes.c_uint64]
    cache = ctypes.POINTER(KVCache)
    L.pa_norm_rope_store.restype = ctypes.c_int
    L.pa_norm_rope_store.argtypes = [P, i64, P, i64, P, i64, ctypes.POINTER(NormRope), P, P, i32,
                                     i32, cache, P, P, P]
    L.pa_prefill_window.restype = ctypes.c_int
    L.pa_prefill_window.argtypes = [P, cache, P, i32, P, P, i32, i32, i32, i32, ctypes.c_float,
                                    i32, i32, P, P]
    L.pa_decode_scored_workspace_size.restype = ctypes.c_size_t
    L.pa_decode_scored_workspace_size.argtypes = [cache, i32, i32, i32, i32]
    L.pa_decode_scored.restype = ctypes.c_int
    L.pa_decode_scored.argtypes = [P, cache, P, i32, P, i32, i32, i32, ctypes.c_float, P, P, P,
                                   ctypes.c_size_t, P]
    L.pa_evict.restype = ctypes.c_int
    L.pa_evict.argtypes = [cache, P, P, i32, P, i32, i32, i32, i32, i32, P, P, P]
    L.pa_norm_rope_axes_store.restype = ctypes.c_int
    L.pa_norm_rope_axes_store.argtypes = [P, i64, P, i64, P, i64, ctypes.POINTER(NormRope), P, i32,
                                          ctypes.c_char_p, P, i32, i32, cache, P, P, P]
    L.pa_decode_shared_workspace_size.restype = ctypes.c_size_t
    L.pa_decode_shared_workspace_size.argtypes = [cache, i32, i32, i32, i32, i32]
    L.pa_decode_shared.restype = ctypes.c_int
    L.pa_decode_shared.argtypes = [P, cache, P, i32, P, i32, P, P, i32, i32, i32, i32,
                                   ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.pa_prefill_shared_workspace_size.restype = ctypes.c_size_t
    L.pa_prefill_shared_workspace_size.argtypes = [cache, i32, i32, i32]
    L.pa_prefill_shared.restype = ctypes.c_int
    L.pa_prefill_shared.argtypes = [P, cache, P, i32, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                    ctypes.c_float, P, P, ctypes.c_size_t, P]
    _lib = L
    return L


def _ptr(t: torch.Tensor | None):
    # a plain int: the prototypes declare c_void_p, which ctypes fills from it
    return None if t is None else t.data_ptr()


# The raw handle of the current stream, without building a torch.cuda.Stream
# object per call (a tenth of the cost; the public call is the fallback).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _check(code: int, what: str):
    if code != 0:
        raise PAError(code, what)


def _state(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: int) -> torch.Tensor:
    """A tensor that a call writes, or reads where it lies: refuse any other type, shape, device
    or layout."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:  # a torch.Size is a tuple
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the caches' device, not on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _input(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: int) -> torch.Tensor:
    """A tensor that a call reads, made contiguous if it is not."""
    if t.is_contiguous():
        return _state(t, name, dtype, shape, dev)
    return _state(t.contiguous(), name, dtype, shape, dev)


def _check_i32(**numbers: int) -> None:
    """Refuse arguments of a C call that do not fit 32 bits: ctypes would drop their upper bits."""
    for name, x in numbers.items():
        if not -0x80000000 <= x <= 0x7fffffff:
            raise ValueError(f"{name} must fit 32 bits, got {x}")


_KV_CODES = {torch.bfloat16: PA_KV_BF16, torch.uint8: PA_KV_FP8_E4M3,
             torch.float8_e4m3fn: PA_KV_FP8_E4M3, torch.int8: PA_KV_INT8}


def _cache_of(k_cache, v_cache, k_scale, v_scale, dev: int) -> KVCache:
    """make_cache of caches that agree with each other, all on device `dev` (-1: not a CUDA
    device, refused)."""
    shape, dtype = k_cache.shape, k_cache.dtype
    code = _KV_CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported cache dtype {dtype}")
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not dtype:
        raise ValueError("k_cache and v_cache must have the same 4-D shape and dtype")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("cache tensors must be contiguous")
    if v_cache.get_device() != dev:
        raise ValueError("k_cache and v_cache must be on the same device")
    nb, bs, hkv, d = shape
    ks = vs = None
    if k_scale is not None or v_scale is not None:
        if k_scale is None or v_scale is None:
            raise ValueError("k_scale and v_scale come together")
        ks = _state(k_scale, "k_scale", torch.float32, (nb, hkv, bs), dev).data_ptr()
        vs = _state(v_scale, "v_scale", torch.float32, (nb, hkv, bs), dev).data_ptr()
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    return KVCache(nb, bs, hkv, d, code, k_cache.data_ptr(), v_cache.data_ptr(), ks, vs)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(device: int, what: str, fn, *args) -> None:
    """fn(*args, stream) on device `device` and its current stream."""
    if device == _current_device():
        code = fn(*args, _raw_stream(device) if _raw_stream is not None else _stream())
    else:
        with torch.cuda.device(device):
            code = fn(*args, _stream())
    if code != 0:
        raise PAError(code, what)


def make_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor | None = None,
               v_scale: torch.Tensor | None = None) -> KVCache:
    """Describe caches of shape (num_blocks, block_size, num_kv_heads, head_dim):
    bf16, or uint8 E4M3 / int8 codes with fp32 scales (num_blocks, num_kv_heads,
    block_size)."""
    if k_cache.dtype == torch.bfloat16:
        dt = PA_KV_BF16
    elif k_cache.dtype in (torch.uint8, torch.float8_e4m3fn):
        dt = PA_KV_FP8_E4M3
    elif k_cache.dtype == torch.int8:
        dt = PA_KV_INT8
    else:
        raise TypeError(f"unsupported cache dtype {k_cache.dtype}")
    for t in (k_cache, v_cache, k_scale, v_scale):
        if t is not None and not t.is_contiguous():
            raise ValueError("cache tensors must be contiguous")
    nb, bs, hkv, d = k_cache.shape
    return KVCache(nb, bs, hkv, d, dt, k_cache.data_ptr(), v_cache.data_ptr(),
                   None if k_scale is None else k_scale.data_ptr(),
                   None if v_scale is None else v_scale.data_ptr())


def store_kv(k, v, slot_mapping, k_cache, v_cache, k_scale_new=None, v_scale_new=None,
             k_scale=None, v_scale=None) -> None:
    """pa_store_kv: write k/v (T, Hkv, D) to their slots (int64 (T,)), in place."""
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    k, v = k.contiguous(), v.contiguous()
    sm = slot_mapping.contiguous()
    _check(lib().pa_store_kv(_ptr(k), _ptr(v), _ptr(k_scale_new), _ptr(v_scale_new), _ptr(sm),
                             int(sm.numel()), ctypes.byref(cache), _stream()), "pa_store_kv")


def decode_workspace_size(k_cache, batch: int, num_heads: int, max_blocks_per_seq: int,
                          max_context_len: int = 0, v_cache=None, k_scale=None,
                          v_scale=None) -> int:
    cache = make_cache(k_cache, k_cache if v_cache is None else v_cache, k_scale, v_scale)
    return int(lib().pa_decode_workspace_size(ctypes.byref(cache), batch, num_heads,
                                              max_blocks_per_seq, max_context_len))


def decode(q, k_cache, v_cache, block_tables, context_lens, scale: float, *,
           max_context_len: int = 0, out=None, workspace=None, k_scale=None,
           v_scale=None) -> torch.Tensor:
    """pa_decode: q (B, H, D) bf16 -> out (B, H, D) bf16.

    max_context_len is the host-side bound of context_lens (0 = block-table
    capacity). A workspace (uint8 tensor) is allocated when none is given.
    """
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    B, H, D = q.shape
    bt = block_tables.contiguous()
    cl = context_lens.contiguous()
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    if workspace is None:  # a caller-provided workspace is checked by the library
        need = int(lib().pa_decode_workspace_size(ctypes.byref(cache), B, H, bt.shape[1],
                                                  max_context_len))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pa_decode(_ptr(q.contiguous()), ctypes.byref(cache), _ptr(bt), bt.shape[1],
                           _ptr(cl), int(max_context_len), B, H, float(scale), _ptr(out),
                           _ptr(workspace), ws_bytes, _stream()), "pa_decode")
    return out


def decode_window(q, k_cache, v_cache, block_tables, context_lens, scale: float, window: int,
                  sinks: int = 0, *, max_context_len: int = 0, out=None, workspace=None,
                  k_scale=None, v_scale=None) -> torch.Tensor:
    """pa_decode_window: decode attention over the last `window` keys and the
    first `sinks` keys of each sequence (window <= 0: all keys)."""
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    B, H, D = q.shape
    bt = block_tables.contiguous()
    cl = context_lens.contiguous()
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    if workspace is None:
        need = int(lib().pa_decode_workspace_size(ctypes.byref(cache), B, H, bt.shape[1],
                                                  max_context_len))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pa_decode_window(_ptr(q.contiguous()), ctypes.byref(cache), _ptr(bt),
                                  bt.shape[1], _ptr(cl), int(max_context_len), B, H, float(scale),
                                  int(window), int(sinks), _ptr(out), _ptr(workspace), ws_bytes,
                                  _stream()), "pa_decode_window")
    return out


def decode_append(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                  scale: float, *, max_context_len: int = 0, out=None, workspace=None,
                  k_scale_new=None, v_scale_new=None, k_scale=None,
                  v_scale=None) -> torch.Tensor:
    """pa_decode_append: write each sequence's new K/V row (k_new/v_new
    (B, Hkv, D), cache dtype) at position context_len-1 through the block
    table, in place, and return decode attention over context_len keys."""
    return decode_window_append(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                                scale, 0, 0, max_context_len=max_context_len, out=out,
                                workspace=workspace, k_scale_new=k_scale_new,
                                v_scale_new=v_scale_new, k_scale=k_scale, v_scale=v_scale)


def decode_window_append(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                         scale: float, window: int, sinks: int = 0, *, max_context_len: int = 0,
                         out=None, workspace=None, k_scale_new=None, v_scale_new=None,
                         k_scale=None, v_scale=None) -> torch.Tensor:
    """pa_decode_window_append (window 0: pa_decode_append): write each
    sequence's new K/V row at position context_len-1 through the block table,
    in place, and return decode attention over the last `window` keys and the
    first `sinks` keys (window <= 0: all context_len keys)."""
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    B, H, D = q.shape
    bt = block_tables.contiguous()
    cl = context_lens.contiguous()
    k_new, v_new = k_new.contiguous(), v_new.contiguous()
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    if workspace is None:
        need = int(lib().pa_decode_workspace_size(ctypes.byref(cache), B, H, bt.shape[1],
                                                  max_context_len))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if int(window) > 0:
        rc = lib().pa_decode_window_append(
            _ptr(q.contiguous()), _ptr(k_new), _ptr(v_new), _ptr(k_scale_new), _ptr(v_scale_new),
            ctypes.byref(cache), _ptr(bt), bt.shape[1], _ptr(cl), int(max_context_len), B, H,
            float(scale), int(window), int(sinks), _ptr(out), _ptr(workspace), ws_bytes,
            _stream())
        _check(rc, "pa_decode_window_append")
    else:
        rc = lib().pa_decode_append(
            _ptr(q.contiguous()), _ptr(k_new), _ptr(v_new), _ptr(k_scale_new), _ptr(v_scale_new),
            ctypes.byref(cache), _ptr(bt), bt.shape[1], _ptr(cl), int(max_context_len), B, H,
            float(scale), _ptr(out), _ptr(workspace), ws_bytes, _stream())
        _check(rc, "pa_decode_append")
    return out


def prefill_varlen(q, k_cache, v_cache, block_tables, cu_seqlens_q, cu_seqlens_k,
                   scale: float, *, max_q_len: int = 0, out=None) -> torch.Tensor:
    """pa_prefill_varlen: packed q (total_q, H, D) bf16 -> out (total_q, H, D) bf16,
    attending over each sequence's paged K/V with the bottom-right causal mask.
    The new tokens' K/V must already be in the cache (store_kv)."""
    cache = make_cache(k_cache, v_cache)
    T, H, D = q.shape
    bt = block_tables.contiguous()
    cq, ck = cu_seqlens_q.contiguous(), cu_seqlens_k.contiguous()
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    _check(lib().pa_prefill_varlen(_ptr(q.contiguous()), ctypes.byref(cache), _ptr(bt),
                                   bt.shape[1], _ptr(cq), _ptr(ck), cq.numel() - 1, H, T,
                                   int(max_q_len), float(scale), _ptr(out), _stream()),
           "pa_prefill_varlen")
    return out


def _token_rows(t: torch.Tensor, name: str, shape, dev: int):
    """(address, element stride between tokens, tensor) of bf16 `shape` = (T, heads, head_dim)
    whose tokens' heads are contiguous: a view of a fused projection's output is taken as it
    is, any other layout is copied."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the caches' device, not on {t.device}")
    T, H, D = shape
    row = H * D
    st, sh, sd = t.stride()
    if T == 1:
        st = row
    p = t.data_ptr()
    if sd != 1 or (sh != D and H > 1) or st < row or st % 8 or p % 16:
        t = t.clone(memory_format=torch.contiguous_format)
        return t.data_ptr(), row, t
    return p, st, t


def norm_rope_store(q, k, v, positions, slot_mapping, k_cache, v_cache, *, q_weight=None,
                    k_weight=None, eps: float = 1e-6, cos_sin=None, interleaved: bool = False,
                    q_out=None, k_scale=None, v_scale=None, scores=None) -> torch.Tensor:
    """pa_norm_rope_store: RMS norm of every head of q (T, H, D) and k (T, Hkv, D) (where its
    bf16 (D,) weight is given), rotation by the row `positions` (int64 (T,)) of cos_sin
    (max_positions, rotary_dim: cosines, then sines; None: no rotation), and the store of k and
    v in their slots (int64 (T,), negative: a padding token, skipped) of the cache, quantised
    for an 8-bit cache. Returns q_out (T, H, D) bf16 (rows of padding tokens are not written);
    it may be q itself if q is contiguous. q, k and v may be views of one fused projection's
    output. scores: set the slots' scores (decode_scored) to 0."""
    return _norm_rope(q, k, v, positions, slot_mapping, k_cache, v_cache, None, q_weight, k_weight,
                      eps, cos_sin, interleaved, q_out, k_scale, v_scale, scores)


def norm_rope_axes_store(q, k, v, positions, slot_mapping, k_cache, v_cache, pair_axis, cos_sin, *,
                         q_weight=None, k_weight=None, eps: float = 1e-6,
                         interleaved: bool = False, q_out=None, k_scale=None, v_scale=None,
                         scores=None) -> torch.Tensor:
    """pa_norm_rope_axes_store: norm_rope_store for tokens with a position on each of one to four
    axes (time, height, width): positions is (axes, T) int64, and pair i of the rotated dims takes
    column i of the table's row positions[pair_axis[i]]. pair_axis: the axis of each of the
    rotary_dim / 2 pairs, as bytes (quickest) or integers, e.g. [0] * 16 + [1] * 24 + [2] * 24."""
    if cos_sin is None or positions is None:
        raise ValueError("norm_rope_axes_store needs cos_sin and positions")
    if positions.dim() != 2:
        raise ValueError("positions must be (axes, tokens)")
    if not isinstance(pair_axis, bytes):
        # (a list: bytes() takes a number for a length and an array for its memory)
        pair_axis = bytes(list(pair_axis))  # refuses what is not 0 .. 255
    return _norm_rope(q, k, v, positions, slot_mapping, k_cache, v_cache, pair_axis, q_weight,
                      k_weight, eps, cos_sin, interleaved, q_out, k_scale, v_scale, scores)


def _norm_rope(q, k, v, positions, slot_mapping, k_cache, v_cache, pair_axis, q_weight, k_weight,
               eps, cos_sin, interleaved, q_out, k_scale, v_scale, scores) -> torch.Tensor:
    """The body of norm_rope_store (pair_axis None) and norm_rope_axes_store."""
    dev = k_cache.get_device()
    NB, bs, Hkv, D = k_cache.shape
    if q.dim() != 3:
        raise ValueError("q must be (tokens, num_heads, head_dim)")
    T, H, _ = q.shape
    qp, qs, qc = _token_rows(q, "q", (T, H, D), dev)
    kp, ks, kc = _token_rows(k, "k", (T, Hkv, D), dev)
    vp, vs, vc = _token_rows(v, "v", (T, Hkv, D), dev)
    slot_mapping = _input(slot_mapping, "slot_mapping", torch.int64, (T,), dev)
    rows = rot = 0
    cp = pp = qw = kw = sp = None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be (max_positions, rotary_dim)")
        rows, rot = cos_sin.shape
        cp = _state(cos_sin, "cos_sin", torch.float32, (rows, rot), dev).data_ptr()
        if positions is None:
            raise ValueError("a rotation needs positions")
    axes = () if pair_axis is None else (positions.shape[0],)
    if positions is not None:
        positions = _input(positions, "positions", torch.int64, axes + (T,), dev)
        pp = positions.data_ptr()
    if pair_axis is not None and len(pair_axis) != rot // 2:
        raise ValueError(f"pair_axis must name {rot // 2} axes, one per pair, got {len(pair_axis)}")
    if q_weight is not None:
        qw = _state(q_weight, "q_weight", torch.bfloat16, (D,), dev).data_ptr()
    if k_weight is not None:
        kw = _state(k_weight, "k_weight", torch.bfloat16, (D,), dev).data_ptr()
    if scores is not None:
        sp = _state(scores, "scores", torch.float32, (NB, Hkv, bs), dev).data_ptr()
    if q_out is None:
        q_out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _state(q_out, "q_out", torch.bfloat16, (T, H, D), dev)
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    params = NormRope(qw, kw, cp, rows, rot, 1 if interleaved else 0, eps)
    if pair_axis is None:
        _run(dev, "pa_norm_rope_store", (_lib or lib()).pa_norm_rope_store, qp, qs, kp, ks, vp, vs,
             ctypes.byref(params), pp, slot_mapping.data_ptr(), T, H, ctypes.byref(cache), sp,
             q_out.data_ptr())
    else:
        _run(dev, "pa_norm_rope_axes_store", (_lib or lib()).pa_norm_rope_axes_store, qp, qs, kp,
             ks, vp, vs, ctypes.byref(params), pp, axes[0], pair_axis, slot_mapping.data_ptr(), T,
             H, ctypes.byref(cache), sp, q_out.data_ptr())
    return q_out


def prefill_window(q, k_cache, v_cache, block_tables, cu_seqlens_q, cu_seqlens_k, scale: float,
                   window: int, sinks: int = 0, *, max_q_len: int = 0,
                   out=None) -> torch.Tensor:
    """pa_prefill_window: prefill_varlen where a query sees the last `window` (>= 1) keys up to
    its own and the first `sinks` keys. bf16 caches of head_dim 128. max_q_len (a bound of every
    sequence's new tokens) lets short continuations take their own variant."""
    if q.dim() != 3:
        raise ValueError("q must be (total_q, num_heads, head_dim)")
    max_q_len, window, sinks = int(max_q_len), int(window), int(sinks)
    if not 0 <= max_q_len | window | sinks <= 0x7fffffff:  # (all of them: one comparison)
        _check_i32(max_q_len=max_q_len, window=window, sinks=sinks)
    dev = k_cache.get_device()
    T, H, D = q.shape
    n = cu_seqlens_q.numel()
    if n < 1 or block_tables.dim() != 2:
        raise ValueError("block_tables must be (batch, blocks), cu_seqlens (batch + 1,)")
    width = block_tables.shape[1]
    q = _input(q, "q", torch.bfloat16, (T, H, k_cache.shape[3]), dev)
    cu_q = _input(cu_seqlens_q, "cu_seqlens_q", torch.int32, (n,), dev)
    cu_k = _input(cu_seqlens_k, "cu_seqlens_k", torch.int32, (n,), dev)
    bt = _input(block_tables, "block_tables", torch.int32, (n - 1, width), dev)
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _state(out, "out", torch.bfloat16, (T, H, D), dev)
    cache = _cache_of(k_cache, v_cache, None, None, dev)
    _run(dev, "pa_prefill_window", (_lib or lib()).pa_prefill_window, q.data_ptr(),
         ctypes.byref(cache), bt.data_ptr(), width, cu_q.data_ptr(), cu_k.data_ptr(), n - 1, H, T,
         max_q_len, scale, window, sinks, out.data_ptr())
    return out


def decode_scored_workspace_size(k_cache, batch: int, num_heads: int, max_blocks_per_seq: int,
                                 max_context_len: int = 0, v_cache=None, k_scale=None,
                                 v_scale=None) -> int:
    """Bytes of the workspace of decode_scored (0: the shape is not supported)."""
    _check_i32(batch=batch, num_heads=num_heads, max_blocks_per_seq=max_blocks_per_seq,
               max_context_len=max_context_len)
    cache = make_cache(k_cache, k_cache if v_cache is None else v_cache, k_scale, v_scale)
    return int(lib().pa_decode_scored_workspace_size(ctypes.byref(cache), batch, num_heads,
                                                     max_blocks_per_seq, max_context_len))


def decode_scored(q, k_cache, v_cache, block_tables, context_lens, scores, scale: float, *,
                  max_context_len: int = 0, out=None, workspace=None, k_scale=None,
                  v_scale=None) -> torch.Tensor:
    """pa_decode_scored: decode, and every visible key's softmax weight, summed over the query
    heads of its kv head, added in place to scores (num_blocks, num_kv_heads, block_size) fp32.
    A workspace (uint8 tensor of decode_scored_workspace_size bytes: four per query head and key
    of the bound) is allocated in every call that gives none."""
    if q.dim() != 3:
        raise ValueError("q must be (batch, num_heads, head_dim)")
    max_context_len = int(max_context_len)
    if not 0 <= max_context_len <= 0x7fffffff:
        _check_i32(max_context_len=max_context_len)
    dev = k_cache.get_device()
    B, H, D = q.shape
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be (batch, blocks)")
    width = block_tables.shape[1]
    nb, bs, hkv, d = k_cache.shape
    q = _input(q, "q", torch.bfloat16, (B, H, d), dev)
    cl = _input(context_lens, "context_lens", torch.int32, (B,), dev)
    bt = _input(block_tables, "block_tables", torch.int32, (B, width), dev)
    _state(scores, "scores", torch.float32, (nb, hkv, bs), dev)
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _state(out, "out", torch.bfloat16, (B, H, D), dev)
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    ws = ws_bytes = 0
    if workspace is None:  # a caller-provided workspace is checked by the library
        need = decode_scored_workspace_size(k_cache, B, H, width, max_context_len, v_cache,
                                            k_scale, v_scale)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be contiguous and on the caches' device")
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _run(dev, "pa_decode_scored", (_lib or lib()).pa_decode_scored, q.data_ptr(),
         ctypes.byref(cache), bt.data_ptr(), width, cl.data_ptr(), max_context_len, B, H,
         scale, scores.data_ptr(), out.data_ptr(), ws or None, ws_bytes)
    return out


def _groups(cu_groups, prefix_lens, dev: int):
    """(cu_groups, prefix_lens, number of groups), checked."""
    n = prefix_lens.numel()
    return (_input(cu_groups, "cu_groups", torch.int32, (n + 1,), dev),
            _input(prefix_lens, "prefix_lens", torch.int32, (n,), dev), n)


def decode_shared_workspace_size(k_cache, batch: int, num_heads: int, max_blocks_per_seq: int,
                                 num_groups: int, max_context_len: int = 0, v_cache=None,
                                 k_scale=None, v_scale=None) -> int:
    """Bytes of the workspace of decode_shared (0: the shape is not supported)."""
    _check_i32(batch=batch, num_heads=num_heads, max_blocks_per_seq=max_blocks_per_seq,
               num_groups=num_groups, max_context_len=max_context_len)
    cache = make_cache(k_cache, k_cache if v_cache is None else v_cache, k_scale, v_scale)
    return int(lib().pa_decode_shared_workspace_size(ctypes.byref(cache), batch, num_heads,
                                                     max_blocks_per_seq, num_groups,
                                                     max_context_len))


def decode_shared(q, k_cache, v_cache, block_tables, context_lens, cu_groups, prefix_lens,
                  scale: float, *, max_context_len: int = 0, always: bool = False, out=None,
                  workspace=None, k_scale=None, v_scale=None) -> torch.Tensor:
    """pa_decode_shared: decode where the sequences cu_groups[g] .. cu_groups[g+1]-1 (int32
    (groups + 1,)) share their first prefix_lens[g] keys (int32 (groups,)): their block table rows
    begin with the same prefix_lens[g] // block_size blocks, which are read and attended to once
    for the whole group (if that would pay were all of max_context_len, or of the table's width,
    shared; always: in any case). Where prefixes are not most of the contexts decode is faster. A
    workspace (uint8 tensor of decode_shared_workspace_size bytes) is allocated in every call that
    gives none."""
    if q.dim() != 3:
        raise ValueError("q must be (batch, num_heads, head_dim)")
    max_context_len = int(max_context_len)
    if not 0 <= max_context_len <= 0x7fffffff:
        _check_i32(max_context_len=max_context_len)
    dev = k_cache.get_device()
    B, H, D = q.shape
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be (batch, blocks)")
    width = block_tables.shape[1]
    q = _input(q, "q", torch.bfloat16, (B, H, k_cache.shape[3]), dev)
    cl = _input(context_lens, "context_lens", torch.int32, (B,), dev)
    bt = _input(block_tables, "block_tables", torch.int32, (B, width), dev)
    cg, pl, n = _groups(cu_groups, prefix_lens, dev)
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _state(out, "out", torch.bfloat16, (B, H, D), dev)
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    ws = ws_bytes = 0
    if workspace is None:  # a caller-provided workspace is checked by the library
        need = decode_shared_workspace_size(k_cache, B, H, width, n, max_context_len, v_cache,
                                            k_scale, v_scale)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be contiguous and on the caches' device")
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _run(dev, "pa_decode_shared", (_lib or lib()).pa_decode_shared, q.data_ptr(),
         ctypes.byref(cache), bt.data_ptr(), width, cl.data_ptr(), max_context_len, cg.data_ptr(),
         pl.data_ptr(), n, 1 if always else 0, B, H, scale, out.data_ptr(), ws or None, ws_bytes)
    return out


def prefill_shared_workspace_size(k_cache, total_q: int, num_heads: int, num_groups: int) -> int:
    """Bytes of the workspace of prefill_shared (0: the shape is not supported)."""
    _check_i32(total_q=total_q, num_heads=num_heads, num_groups=num_groups)
    cache = make_cache(k_cache, k_cache)
    return int(lib().pa_prefill_shared_workspace_size(ctypes.byref(cache), num_heads, total_q,
                                                      num_groups))


def prefill_shared(q, k_cache, v_cache, block_tables, cu_seqlens_q, cu_seqlens_k, cu_groups,
                   prefix_lens, scale: float, *, max_q_len: int = 0, always: bool = False,
                   out=None, workspace=None) -> torch.Tensor:
    """pa_prefill_shared: prefill_varlen of sequences that share their first keys in groups
    (cu_groups, prefix_lens, always: as decode_shared). bf16 caches of head_dim 128. max_q_len (a bound of
    every sequence's new tokens) sizes the grid and lets short questions take their own variant. A
    workspace (uint8 tensor of prefill_shared_workspace_size bytes: about 8 * head_dim a query row and
    head, and some MB for the groups and the SMs) is allocated in every call that gives none."""
    if q.dim() != 3:
        raise ValueError("q must be (total_q, num_heads, head_dim)")
    max_q_len = int(max_q_len)
    if not 0 <= max_q_len <= 0x7fffffff:
        _check_i32(max_q_len=max_q_len)
    dev = k_cache.get_device()
    T, H, D = q.shape
    n = cu_seqlens_q.numel()
    if n < 1 or block_tables.dim() != 2:
        raise ValueError("block_tables must be (batch, blocks), cu_seqlens (batch + 1,)")
    width = block_tables.shape[1]
    q = _input(q, "q", torch.bfloat16, (T, H, k_cache.shape[3]), dev)
    cu_q = _input(cu_seqlens_q, "cu_seqlens_q", torch.int32, (n,), dev)
    cu_k = _input(cu_seqlens_k, "cu_seqlens_k", torch.int32, (n,), dev)
    bt = _input(block_tables, "block_tables", torch.int32, (n - 1, width), dev)
    cg, pl, groups = _groups(cu_groups, prefix_lens, dev)
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _state(out, "out", torch.bfloat16, (T, H, D), dev)
    cache = _cache_of(k_cache, v_cache, None, None, dev)
    ws = ws_bytes = 0
    if workspace is None:  # a caller-provided workspace is checked by the library
        need = prefill_shared_workspace_size(k_cache, T, H, groups)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be contiguous and on the caches' device")
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _run(dev, "pa_prefill_shared", (_lib or lib()).pa_prefill_shared, q.data_ptr(),
         ctypes.byref(cache), bt.data_ptr(), width, cu_q.data_ptr(), cu_k.data_ptr(),
         cg.data_ptr(), pl.data_ptr(), groups, 1 if always else 0, n - 1, H, T, max_q_len, scale,
         out.data_ptr(), ws or None, ws_bytes)
    return out


def evict(k_cache, v_cache, scores, block_tables, context_lens, budget: int, *, sinks: int = 0,
          recent: int = 0, max_context_len: int = 0, kept=None, new_lens=None, k_scale=None,
          v_scale=None) -> tuple[torch.Tensor, torch.Tensor]:
    """pa_evict: cut every sequence of more than `budget` keys to, per kv head, its first
    `sinks`, its last `recent` and the best scores between them, moved in order to the front of
    its blocks (K, V, scales and scores, in place). Returns (new_lens (B,) int32,
    kept (B, Hkv, budget) int32: the positions the rows came from). Pass max_context_len where
    the block table is much wider than the sequences: it sizes the selection."""
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    max_context_len = int(max_context_len)
    if not 0 <= budget | sinks | recent | max_context_len <= 0x7fffffff:
        _check_i32(budget=budget, sinks=sinks, recent=recent, max_context_len=max_context_len)
    dev = scores.get_device()
    B = context_lens.numel()
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be (batch, blocks)")
    width = block_tables.shape[1]
    nb, bs, hkv, _ = k_cache.shape
    cl = _input(context_lens, "context_lens", torch.int32, (B,), dev)
    bt = _input(block_tables, "block_tables", torch.int32, (B, width), dev)
    _state(scores, "scores", torch.float32, (nb, hkv, bs), dev)
    if kept is None:
        kept = torch.empty((B, hkv, max(budget, 0)), dtype=torch.int32, device=scores.device)
    else:
        _state(kept, "kept", torch.int32, (B, hkv, budget), dev)
    if new_lens is None:
        new_lens = torch.empty((B,), dtype=torch.int32, device=scores.device)
    else:
        _state(new_lens, "new_lens", torch.int32, (B,), dev)
    if k_cache.get_device() != dev:
        raise ValueError("k_cache must be on the scores' device")
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    _run(dev, "pa_evict", (_lib or lib()).pa_evict, ctypes.byref(cache), scores.data_ptr(),
         bt.data_ptr(), width, cl.data_ptr(), max_context_len, B, budget, sinks,
         recent, kept.data_ptr(), new_lens.data_ptr())
    return new_lens, kept


def decode_noalloc(q, k_cache, v_cache, block_tables, context_lens, scale: float, *,
                   max_context_len: int = 0, out=None, k_scale=None,
                   v_scale=None) -> torch.Tensor:
    """pa_decode_noalloc: pa_decode with the split-K scratch taken from the
    library's static device buffer instead of a caller workspace. For callers
    that cannot allocate device memory; `out` should then be passed in."""
    cache = make_cache(k_cache, v_cache, k_scale, v_scale)
    B, H, D = q.shape
    bt = block_tables.contiguous()
    cl = context_lens.contiguous()
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    _check(lib().pa_decode_noalloc(_ptr(q.contiguous()), ctypes.byref(cache), _ptr(bt),
                                   bt.shape[1], _ptr(cl), int(max_context_len), B, H,
                                   float(scale), _ptr(out), _stream()), "pa_decode_noalloc")
    return out


def debug_inject_wait_timeout(skip_copy: int, wait_limit_ns: int = 0) -> None:
    """pa_debug_inject_wait_timeout: arm (skip_copy >= 0) or disarm (< 0) the
    failure-detection test hook of the decode kernels."""
    _check(lib().pa_debug_inject_wait_timeout(int(skip_copy), int(wait_limit_ns)),
           "pa_debug_inject_wait_timeout")


def get_device_error() -> int:
    """Synchronise the device, return and clear its PA_DEVERR_* word."""
    code = ctypes.c_uint32(0)
    _check(lib().pa_get_device_error(ctypes.byref(code)), "pa_get_device_error")
    return int(code.value)

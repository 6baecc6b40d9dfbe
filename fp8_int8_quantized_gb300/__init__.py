"""Python binding of the kvq C ABI (``include/kvq.h``): a GB300 quantized paged
KV cache -- FP8 (E4M3 / E5M2, per-tensor scale) or online INT8 / INT4
(one scale per row or per channel group) quantize-on-write -- with single-token
decode attention (optionally fused with the step's append) and chunked causal
prefill attention that dequantize on read; and for speculative serving, append
with the position rotation of Q and K, attention of a few draft tokens per
sequence (a chain or a tree) and moves of cached rows.

This module only marshals arguments: it checks tensor dtypes, devices and
layouts, passes raw device pointers and the current CUDA stream to
``libkvq.so`` and raises on a non-OK status.  Every step of the hot path runs in
the library's CUDA kernels.  PyTorch supplies device memory and streams.  There
is no CPU fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

E4M3, E5M2, INT8, INT4 = 1, 2, 3, 4
FORMATS = {"e4m3": E4M3, "fp8": E4M3, "e5m2": E5M2, "fp8_e5m2": E5M2, "int8": INT8, "int4": INT4}
STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED", 3: "KVQ_ERR_WORKSPACE",
          4: "KVQ_ERR_OUT_OF_RANGE", 5: "KVQ_ERR_TIMEOUT", 6: "KVQ_ERR_CUDA",
          7: "KVQ_ERR_SCRATCH_LIMIT"}
KERNEL_AUTO, KERNEL_SIMT, KERNEL_MMA = 0, 1, 2
EXPORTS = ("kvq_append", "kvq_decode_workspace_size", "kvq_decode_attention", "kvq_decode_attention_append",
           "kvq_dequant",
           "kvq_set_decode_kernel", "kvq_device_error_check", "kvq_status_string", "kvq_abi_version",
           "kvq_decode_attention_static_scratch", "kvq_static_scratch_bytes", "kvq_set_decode_timing_events",
           "kvq_prefill_attention", "kvq_encode_fp8", "kvq_append_rotary", "kvq_verify_workspace_size",
           "kvq_verify_attention", "kvq_move_rows")

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")
_lib = None
_lock = threading.Lock()


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class KvqCacheDesc(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("fmt", ctypes.c_int32), ("group_size", ctypes.c_int32)]


def build(force: bool = False) -> str:
    from . import build_lib
    return build_lib.build(force=force)


def lib():
    """The loaded ``libkvq.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run fp8_int8_quantized_gb300.build() first "
                               "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.kvq_append.restype = ctypes.c_int
        L.kvq_append.argtypes = [P, P, P, P, i64, P, i32, P]
        L.kvq_decode_workspace_size.restype = ctypes.c_size_t
        L.kvq_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.kvq_decode_attention.restype = ctypes.c_int
        L.kvq_decode_attention.argtypes = [P, P, P, i32, P, i32, i32, i32, P, i32, ctypes.c_float, P, P,
                                           ctypes.c_size_t, i32, P]
        L.kvq_decode_attention_append.restype = ctypes.c_int
        L.kvq_decode_attention_append.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, P, i32, ctypes.c_float, P,
                                                  P, ctypes.c_size_t, i32, P]
        L.kvq_decode_attention_static_scratch.restype = ctypes.c_int
        L.kvq_decode_attention_static_scratch.argtypes = [P, P, P, i32, P, i32, i32, i32, P, i32, ctypes.c_float,
                                                          P, i32, P]
        L.kvq_static_scratch_bytes.restype = ctypes.c_size_t
        L.kvq_prefill_attention.restype = ctypes.c_int
        L.kvq_prefill_attention.argtypes = [P, P, P, i32, P, P, i32, i64, i32, i32, P, i32, ctypes.c_float, P,
                                            P]
        L.kvq_encode_fp8.restype = ctypes.c_int
        L.kvq_encode_fp8.argtypes = [P, P, i64, i32, P]
        L.kvq_append_rotary.restype = ctypes.c_int
        L.kvq_append_rotary.argtypes = [P, i64, P, i64, P, i64, i32, i32, P, P, i64, P, i32, P, P, i64, i32, i32, P, i32,
                                        P, i64, P]
        L.kvq_verify_workspace_size.restype = ctypes.c_size_t
        L.kvq_verify_workspace_size.argtypes = [i32] * 7
        L.kvq_verify_attention.restype = ctypes.c_int
        L.kvq_verify_attention.argtypes = [P, P, P, i32, P, P, P, i32, i64, i32, i32, i32, P, i32, ctypes.c_float, P, P,
                                           ctypes.c_size_t, P]
        L.kvq_move_rows.restype = ctypes.c_int
        L.kvq_move_rows.argtypes = [P, P, P, P, i32, i64, i32, i32, P]
        L.kvq_dequant.restype = ctypes.c_int
        L.kvq_dequant.argtypes = [P, P, i64, P, i32, P, P, P]
        L.kvq_set_decode_timing_events.restype = None
        L.kvq_set_decode_timing_events.argtypes = [P, P]
        L.kvq_set_decode_kernel.restype = i32
        L.kvq_set_decode_kernel.argtypes = [i32]
        L.kvq_device_error_check.restype = ctypes.c_int
        L.kvq_device_error_check.argtypes = [P, ctypes.POINTER(i64)]
        L.kvq_status_string.restype = ctypes.c_char_p
        L.kvq_status_string.argtypes = [ctypes.c_int]
        L.kvq_abi_version.restype = i32
        _lib = L
        return L


def status_string(status: int) -> str:
    try:
        return lib().kvq_status_string(status).decode()
    except Exception:  # pragma: no cover
        return "?"


def _check(status: int, where: str) -> None:
    if status != 0:
        raise KvqError(status, where)


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _scale_ptr(scale) -> int | None:
    if scale is None:
        return None
    return _dev(scale, torch.float32, "scale")


class KVCache:
    """A paged quantized cache in device memory:
    codes uint8 [num_blocks][num_kv_heads][block_size][head_dim] for K and V
    ([..][head_dim / 2] packed codes for INT4), and for INT8 / INT4 the fp32
    scales [num_blocks][num_kv_heads][block_size] (one per row, group_size 0) or
    [num_blocks][num_kv_heads][block_size][head_dim / group_size] (one per group
    of channels; group_size head_dim / 2 or head_dim / 4)."""

    def __init__(self, num_blocks, num_kv_heads, block_size, head_dim, fmt, device="cuda", fill=None,
                 group_size=0):
        self.fmt = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
        self.num_blocks, self.num_kv_heads = int(num_blocks), int(num_kv_heads)
        self.block_size, self.head_dim = int(block_size), int(head_dim)
        self.group_size = int(group_size)
        shape = (self.num_blocks, self.num_kv_heads, self.block_size,
                 self.head_dim // 2 if self.fmt == INT4 else self.head_dim)
        mk = (lambda: torch.full(shape, fill, dtype=torch.uint8, device=device)) if fill is not None else \
            (lambda: torch.empty(shape, dtype=torch.uint8, device=device))
        self.k_codes, self.v_codes = mk(), mk()
        if self.fmt in (INT8, INT4):
            sshape = shape[:3] + ((self.head_dim // self.group_size,) if self.group_size else ())
            self.k_scales = torch.zeros(sshape, dtype=torch.float32, device=device)
            self.v_scales = torch.zeros(sshape, dtype=torch.float32, device=device)
        else:
            self.k_scales = self.v_scales = None
        self._desc = None

    def desc(self) -> KvqCacheDesc:
        """A new C descriptor of this cache."""
        return KvqCacheDesc(self.k_codes.data_ptr(), self.v_codes.data_ptr(),
                            self.k_scales.data_ptr() if self.k_scales is not None else None,
                            self.v_scales.data_ptr() if self.v_scales is not None else None,
                            self.num_blocks, self.block_size, self.num_kv_heads, self.head_dim, self.fmt,
                            self.group_size)

    def _cdesc(self) -> KvqCacheDesc:
        # the binding's own descriptor, built once per format (the arrays never move)
        if self._desc is None or self._desc.fmt != self.fmt:
            self._desc = self.desc()
        return self._desc


def append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, slot_mapping: torch.Tensor,
           scale: torch.Tensor | None = None, stream=None) -> None:
    """kvq_append: quantize fp16 K/V [T][Hkv][D] into ``cache`` at ``slot_mapping`` (int64, -1 skips)."""
    T = slot_mapping.shape[0]
    if k.shape != (T, cache.num_kv_heads, cache.head_dim) or v.shape != k.shape:
        raise ValueError("k/v must be [num_tokens][num_kv_heads][head_dim]")
    d = cache._cdesc()
    st = lib().kvq_append(_dev(k, torch.float16, "k"), _dev(v, torch.float16, "v"), ctypes.byref(d),
                          _dev(slot_mapping, torch.int64, "slot_mapping"), T, _scale_ptr(scale), cache.fmt,
                          _stream(stream))
    _check(st, "kvq_append")


def workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, partition_size=0) -> int:
    return int(lib().kvq_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                               max_context_len, partition_size))


def decode_attention(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor, context_lens: torch.Tensor,
                     max_context_len: int, scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     partition_size: int = 0, stream=None) -> torch.Tensor:
    """kvq_decode_attention: q fp16 [B][Hq][D] -> out fp16 [B][Hq][D]."""
    B, Hq, D = q.shape
    if D != cache.head_dim:
        raise ValueError("head_dim mismatch")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:  # a caller-given workspace is checked by the library
        need = workspace_size(B, Hq, cache.num_kv_heads, D, max_context_len, partition_size)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    d = cache._cdesc()
    st = lib().kvq_decode_attention(_dev(q, torch.float16, "q"), ctypes.byref(d),
                                    _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                    _dev(context_lens, torch.int32, "context_lens"), B, Hq, int(max_context_len),
                                    _scale_ptr(scale), cache.fmt, float(sm_scale),
                                    _dev(out, torch.float16, "out"), ws_ptr, ws_bytes, int(partition_size),
                                    _stream(stream))
    _check(st, "kvq_decode_attention")
    return out


def prefill_attention(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor, context_lens: torch.Tensor,
                      query_start: torch.Tensor, max_query_len: int, scale: torch.Tensor | None = None,
                      sm_scale: float = 0.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_prefill_attention: causal attention of chunks of new queries over the cache.

    q fp16 [Tq][Hq][D]; sequence b owns rows query_start[b] .. query_start[b+1]-1, the last
    positions of its context_lens[b] cached tokens.  Returns out fp16 [Tq][Hq][D]."""
    Tq, Hq, D = q.shape
    if D != cache.head_dim:
        raise ValueError("head_dim mismatch")
    B = context_lens.shape[0]
    if query_start.shape[0] != B + 1:
        raise ValueError("query_start needs batch + 1 entries")
    if out is None:
        out = torch.empty_like(q)
    d = cache._cdesc()
    st = lib().kvq_prefill_attention(_dev(q, torch.float16, "q"), ctypes.byref(d),
                                     _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                     _dev(context_lens, torch.int32, "context_lens"),
                                     _dev(query_start, torch.int32, "query_start"), B, Tq, Hq,
                                     int(max_query_len),
                                     _scale_ptr(scale), cache.fmt, float(sm_scale),
                                     _dev(out, torch.float16, "out"), _stream(stream))
    _check(st, "kvq_prefill_attention")
    return out


def decode_attention_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: KVCache,
                            block_tables: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                            scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            partition_size: int = 0, stream=None) -> torch.Tensor:
    """kvq_decode_attention_append: one decode step with each sequence's newest
    K/V row (fp16 [B][Hkv][D], position context_lens[b] - 1) quantized into the
    cache in the same launch; bit-identical to ``append`` then ``decode_attention``."""
    B, Hq, D = q.shape
    if k_new.shape != (B, cache.num_kv_heads, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [batch][num_kv_heads][head_dim]")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = workspace_size(B, Hq, cache.num_kv_heads, D, max_context_len, partition_size)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    d = cache._cdesc()
    st = lib().kvq_decode_attention_append(_dev(q, torch.float16, "q"), _dev(k_new, torch.float16, "k_new"),
                                           _dev(v_new, torch.float16, "v_new"), ctypes.byref(d),
                                           _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                           _dev(context_lens, torch.int32, "context_lens"), B, Hq,
                                           int(max_context_len), _scale_ptr(scale), cache.fmt, float(sm_scale),
                                           _dev(out, torch.float16, "out"), ws_ptr, ws_bytes, int(partition_size),
                                           _stream(stream))
    _check(st, "kvq_decode_attention_append")
    return out


def decode_attention_static_scratch(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor,
                                    context_lens: torch.Tensor, max_context_len: int,
                                    scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                                    out: torch.Tensor | None = None, partition_size: int = 0,
                                    stream=None) -> torch.Tensor:
    """kvq_decode_attention_static_scratch: decode attention for callers that cannot
    allocate device memory; the split workspace comes from the library's fixed
    device array.  ``out`` must be supplied by such callers."""
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    d = cache._cdesc()
    st = lib().kvq_decode_attention_static_scratch(
        _dev(q, torch.float16, "q"), ctypes.byref(d), _dev(block_tables, torch.int32, "block_tables"),
        block_tables.shape[1], _dev(context_lens, torch.int32, "context_lens"), B, Hq, int(max_context_len),
        _scale_ptr(scale), cache.fmt, float(sm_scale), _dev(out, torch.float16, "out"), int(partition_size),
        _stream(stream))
    _check(st, "kvq_decode_attention_static_scratch")
    return out


# The calls below check their tensors inline and in one condition each: the
# binding's own time is most of a small call's.
def _raw_stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)   # looked up on use: a torch built without CUDA has no such name


def _refuse(t, dtype, name: str, device: int, shape=None) -> None:
    """Says what is wrong with a tensor that a call's condition refused."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on cuda:{device}, the cache's device, got {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous" if shape is None or t.dim() != 3 else
                     f"{name}: the heads of a token must be contiguous, its tokens at least a row apart")


def _ptr(t, dtype, name: str, device: int) -> int:
    """The pointer of a contiguous tensor on the cache's device."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _refuse(t, dtype, name, device)
    return t.data_ptr()


def _rows(t, dtype, name: str, device: int, T: int, heads: int, head_dim: int) -> tuple[int, int]:
    """(pointer, token stride) of rows [T][heads][head_dim] whose heads are contiguous."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != (T, heads, head_dim):
        _refuse(t, dtype, name, device, (T, heads, head_dim))
    row, head, one = t.stride()
    if one != 1 or (head != head_dim and heads > 1):
        _refuse(t, dtype, name, device, (T, heads, head_dim))
    return t.data_ptr(), row if T > 1 else heads * head_dim   # the stride of one token says nothing


def _device_of(cache: KVCache) -> int:
    """The cache's device index (-1: not on a GPU)."""
    return cache.k_codes.get_device()


def _on(device: int, stream, call):
    """call(stream handle) with the cache's device current; with a stream given, on it (what the call
    allocates then belongs to that stream)."""
    if device < 0:
        raise TypeError("the cache is not on a CUDA device")
    if stream is not None and stream.device.index != device:
        raise ValueError(f"stream: expected one of cuda:{device}, the cache's device, got {stream.device}")
    if stream is None and device == torch._C._cuda_getDevice():
        return call(_raw_stream(device))
    with torch.cuda.device(device), torch.cuda.stream(stream):   # (stream None: the current one)
        return call(_raw_stream(device))


def append_rotary(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: KVCache,
                  slot_mapping: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                  scale: torch.Tensor | None = None, axis_of_pair: torch.Tensor | None = None,
                  interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """kvq_append_rotary: rotate Q and K by their positions, quantize K and V into the cache.

    q [T][Hq][D] (or None), k and v [T][Hkv][D], all fp16 or all bf16, views with contiguous
    heads (such as the parts of a fused QKV buffer); positions int64 [T] or [axes][T]; cos_sin
    fp32 [max_position][rot_dim] (cosines, then sines); axis_of_pair uint8 [rot_dim / 2].
    Returns the rotated Q in fp16 (``q_out``; padding rows, slot -1, are left as they were)."""
    dev, T, D, Hkv, dt = _device_of(cache), slot_mapping.shape[0], cache.head_dim, cache.num_kv_heads, k.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise TypeError(f"k: expected float16 or bfloat16, got {dt}")
    kp, ks = _rows(k, dt, "k", dev, T, Hkv, D)
    vp, vs = _rows(v, dt, "v", dev, T, Hkv, D)
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    if positions.shape[-1] != T or positions.dim() > 2:
        raise ValueError("positions must be [num_tokens] or [axes][num_tokens]")
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position][rot_dim]")
    rows, rot = cos_sin.shape
    if axis_of_pair is not None and axis_of_pair.shape != (rot // 2,):
        raise ValueError("axis_of_pair needs one entry per pair")
    Hq = qp = qs = 0
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else 0
        qp, qs = _rows(q, dt, "q", dev, T, Hq, D)
    sp, pp = _ptr(slot_mapping, torch.int64, "slot_mapping", dev), _ptr(positions, torch.int64, "positions", dev)
    tp = _ptr(cos_sin, torch.float32, "cos_sin", dev)
    ap = None if axis_of_pair is None else _ptr(axis_of_pair, torch.uint8, "axis_of_pair", dev)
    cp = None if scale is None else _ptr(scale, torch.float32, "scale", dev)

    def call(s):
        out, op, os_ = q_out, None, 0
        if q is not None:
            if out is None:
                out = torch.empty((T, Hq, D), dtype=torch.float16, device=k.device)
            op, os_ = _rows(out, torch.float16, "q_out", dev, T, Hq, D)
        st = lib().kvq_append_rotary(qp, qs, kp, ks, vp, vs, dt is torch.bfloat16, Hq, ctypes.byref(cache._cdesc()), sp, T, pp,
                                     axes, ap, tp, rows, rot, bool(interleaved), cp, cache.fmt, op, os_, s)
        if st:
            raise KvqError(st, "kvq_append_rotary")
        return out

    return _on(dev, stream, call)


def verify_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_query_len, max_context_len, fmt) -> int:
    return int(lib().kvq_verify_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_query_len,
                                               max_context_len, FORMATS[fmt] if isinstance(fmt, str) else int(fmt)))


@functools.lru_cache(maxsize=512)
def _verify_workspace(device: int, *sizes) -> int:
    """Bytes for these sizes on the current device (its index is part of the key)."""
    return lib().kvq_verify_workspace_size(*sizes)


def verify_attention(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor, context_lens: torch.Tensor,
                     query_start: torch.Tensor, max_query_len: int, max_context_len: int,
                     tree_mask: torch.Tensor | None = None, scale: torch.Tensor | None = None, sm_scale: float = 0.0,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """kvq_verify_attention: attention of 1 to 64 new tokens per sequence over the whole cache.

    q fp16 [Tq][Hq][D]; sequence b owns rows query_start[b] .. query_start[b+1]-1, the last
    positions of its context_lens[b] cached tokens.  tree_mask int64 [Tq]: bit j lets a query see
    the sequence's new token j (itself and its ancestors, in a tree of drafts); None is causal.
    Returns out fp16 [Tq][Hq][D]."""
    dev, (Tq, Hq, D) = _device_of(cache), q.shape
    if D != cache.head_dim:
        raise ValueError("head_dim mismatch")
    B, blocks = block_tables.shape
    if context_lens.shape != (B,) or query_start.shape != (B + 1,):
        raise ValueError("context_lens needs batch entries, query_start batch + 1 and block_tables a row per sequence")
    if tree_mask is not None and tree_mask.shape != (Tq,):
        raise ValueError("tree_mask needs one entry per query")
    if out is not None and out.shape != q.shape:
        raise ValueError("out must have q's shape")
    qp, bp = _ptr(q, torch.float16, "q", dev), _ptr(block_tables, torch.int32, "block_tables", dev)
    lp, sp = _ptr(context_lens, torch.int32, "context_lens", dev), _ptr(query_start, torch.int32, "query_start", dev)
    mp = None if tree_mask is None else _ptr(tree_mask, torch.int64, "tree_mask", dev)
    cp = None if scale is None else _ptr(scale, torch.float32, "scale", dev)

    def call(s):
        o, ws, L = out, workspace, lib()
        if o is None:
            o = torch.empty_like(q)
        op = _ptr(o, torch.float16, "out", dev)
        if ws is None:  # a caller-given workspace is checked by the library
            ws = torch.empty(_verify_workspace(dev, B, Hq, cache.num_kv_heads, D, max_query_len, max_context_len, cache.fmt),
                             dtype=torch.uint8, device=q.device)
        elif ws.get_device() != dev:
            raise ValueError(f"workspace: expected a tensor on cuda:{dev}")
        st = L.kvq_verify_attention(qp, ctypes.byref(cache._cdesc()), bp, blocks, lp, sp, mp, B, Tq, Hq, max_query_len,
                                    max_context_len, cp, cache.fmt, sm_scale, op, ws.data_ptr(),
                                    ws.numel() * ws.element_size(), s)
        if st:
            raise KvqError(st, "kvq_verify_attention")
        return o

    return _on(dev, stream, call)


def move_rows(cache: KVCache, src_slots: torch.Tensor, dst_slots: torch.Tensor, move_start: torch.Tensor,
              max_moves: int, stream=None) -> None:
    """kvq_move_rows: cached row dst_slots[i] <- src_slots[i] (int64), bit for bit; sequence b owns moves
    move_start[b] .. move_start[b+1]-1 (int32, at most ``max_moves`` <= 64 each), all of them read
    before any is written."""
    dev = _device_of(cache)
    if src_slots.dim() != 1 or src_slots.shape != dst_slots.shape or move_start.dim() != 1 or not move_start.shape[0]:
        raise ValueError("src_slots and dst_slots need the same length, move_start batch + 1 entries")
    sp, dp = _ptr(src_slots, torch.int64, "src_slots", dev), _ptr(dst_slots, torch.int64, "dst_slots", dev)
    mp = _ptr(move_start, torch.int32, "move_start", dev)

    def call(s):
        st = lib().kvq_move_rows(ctypes.byref(cache._cdesc()), sp, dp, mp, move_start.shape[0] - 1, src_slots.shape[0], max_moves,
                                 cache.fmt, s)
        if st:
            raise KvqError(st, "kvq_move_rows")

    _on(dev, stream, call)


def dequant(cache: KVCache, slots: torch.Tensor, scale: torch.Tensor | None = None, stream=None):
    """kvq_dequant: fp32 K, V rows [n][Hkv][D] at ``slots`` (int64)."""
    n = slots.shape[0]
    ok = torch.empty((n, cache.num_kv_heads, cache.head_dim), dtype=torch.float32, device=slots.device)
    ov = torch.empty_like(ok)
    d = cache._cdesc()
    st = lib().kvq_dequant(ctypes.byref(d), _dev(slots, torch.int64, "slots"), n, _scale_ptr(scale), cache.fmt,
                           ok.data_ptr(), ov.data_ptr(), _stream(stream))
    _check(st, "kvq_dequant")
    return ok, ov


def encode_fp8(x: torch.Tensor, fmt: int, stream=None) -> torch.Tensor:
    """kvq_encode_fp8: uint8 FP8 codes (``fmt`` E4M3 or E5M2) of a flat fp32 tensor."""
    n = x.numel()
    codes = torch.empty(n, dtype=torch.uint8, device=x.device)
    st = lib().kvq_encode_fp8(_dev(x, torch.float32, "x"), codes.data_ptr(), n, fmt, _stream(stream))
    _check(st, "kvq_encode_fp8")
    return codes


def set_decode_kernel(kind: int) -> int:
    prev = lib().kvq_set_decode_kernel(int(kind))
    if prev < 0:
        raise ValueError(f"unknown decode kernel kind {kind}")
    return prev


def set_decode_timing_events(begin=None, end=None) -> None:
    """kvq_set_decode_timing_events with two recorded torch.cuda.Event objects
    (enable_timing=True), or no arguments to turn the hook off."""
    if begin is None or end is None:
        lib().kvq_set_decode_timing_events(None, None)
    else:
        lib().kvq_set_decode_timing_events(begin.cuda_event, end.cuda_event)


def device_error_check(stream=None) -> tuple[int, int]:
    """(status, detail) of the device error word; synchronizes the stream and clears it."""
    detail = ctypes.c_int64(0)
    st = lib().kvq_device_error_check(_stream(stream), ctypes.byref(detail))
    return st, detail.value

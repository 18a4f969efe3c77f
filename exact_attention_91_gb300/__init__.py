"""Python binding of libfa.so, the GB300 (sm_103a) exact-attention forward.

The C entry points (``include/fa.h``) are exposed under the same names and
take raw device pointers (ints), exactly like the C ABI. ``attention_forward``
is a convenience wrapper for torch tensors: it checks dtypes and layout,
allocates the outputs with torch and calls ``fa_fwd`` on the current stream.
Every step of the computation runs in the CUDA library; if the library is
missing this module raises instead of computing anything elsewhere.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import typing

from .build import LIB_PATH

__all__ = ["FaError", "load_library", "fa_fwd", "fa_fwd_noalloc", "fa_strerror", "fa_device_status",
           "fa_set_wait_limit_ns", "fa_abi_version", "fa_selftest_wait_timeout", "fa_fwd_varlen",
           "fa_varlen_num_splits", "fa_selftest_exp2", "fa_selftest_ex2_rate", "EX2_RATE_THREADS",
           "EX2_RATE_CHAINS", "attention_forward", "attention_forward_varlen",
           "head_shards", "attention_forward_heads", "EXPORTED_SYMBOLS", "CACHE_BF16", "CACHE_E4M3",
           "FaPagedCache", "fa_decode_paged", "fa_decode_paged_workspace", "fa_rotary", "fa_cache_append",
           "fa_page_maps", "attention_decode_paged", "rotary", "rotary_inv_freq", "cache_append", "page_maps",
           "PageMaps"]

EXPORTED_SYMBOLS = ("fa_fwd", "fa_fwd_noalloc", "fa_fwd_varlen", "fa_strerror", "fa_device_status",
                    "fa_set_wait_limit_ns", "fa_abi_version", "fa_selftest_wait_timeout", "fa_varlen_num_splits",
                    "fa_selftest_exp2", "fa_selftest_ex2_rate", "fa_decode_paged", "fa_decode_paged_workspace",
                    "fa_rotary", "fa_cache_append", "fa_page_maps")

FA_OK = 0
FA_ERR_DEVICE_TIMEOUT = -8

# element types of a paged cache
CACHE_BF16 = 0
CACHE_E4M3 = 1

_lib = None


class FaPagedCache(ctypes.Structure):
    """The C ``fa_paged_cache``: one layer's keys and values in pages (device
    pointers, strides in elements)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_block", ctypes.c_longlong), ("k_token", ctypes.c_longlong),
                ("k_head", ctypes.c_longlong), ("v_block", ctypes.c_longlong), ("v_token", ctypes.c_longlong),
                ("v_head", ctypes.c_longlong), ("type", ctypes.c_int), ("num_blocks", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads", ctypes.c_int), ("d", ctypes.c_int)]


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = "fa_fwd"):
        self.status = status
        super().__init__(f"{what} failed: {status} ({fa_strerror(status)})")


def load_library(path: str | None = None):
    """Loads libfa.so (built in-tree by ``exact_attention_91_gb300.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError(
            f"{p} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
    lib = ctypes.CDLL(p)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_noalloc.restype = i
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_strerror.argtypes = [i]
    lib.fa_strerror.restype = ctypes.c_char_p
    lib.fa_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.fa_device_status.restype = i
    lib.fa_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.fa_set_wait_limit_ns.restype = None
    lib.fa_abi_version.argtypes = []
    lib.fa_abi_version.restype = i
    lib.fa_selftest_wait_timeout.argtypes = [vp, ctypes.c_ulonglong]
    lib.fa_selftest_wait_timeout.restype = i
    lib.fa_varlen_num_splits.argtypes = [i, i, i, i, i]
    lib.fa_varlen_num_splits.restype = i
    lib.fa_selftest_exp2.argtypes = [vp, vp, vp, i, vp]
    lib.fa_selftest_exp2.restype = i
    lib.fa_selftest_ex2_rate.argtypes = [vp, vp, i, i, vp]
    lib.fa_selftest_ex2_rate.restype = i
    ll = ctypes.c_longlong
    lib.fa_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, ll, f, vp, ctypes.c_size_t, vp]
    lib.fa_decode_paged.restype = i
    lib.fa_decode_paged_workspace.argtypes = [i] * 8
    lib.fa_decode_paged_workspace.restype = ll
    lib.fa_rotary.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, vp, ll, i, i, i, f, vp]
    lib.fa_rotary.restype = i
    lib.fa_cache_append.argtypes = [vp, vp, vp, ll, ll, ll, vp, vp, vp, vp, vp, vp, ll, ll, i, i, i, i, f, vp]
    lib.fa_cache_append.restype = i
    lib.fa_page_maps.argtypes = [vp] * 9 + [i, i, ll, i, i, i, vp]
    lib.fa_page_maps.restype = i
    if path is None:
        _lib = lib
    return lib


def fa_fwd(q: int, k: int, v: int, o: int, lse: int | None, B: int, H: int, N: int, d: int,
           scale: float, causal: bool, stream: int | None) -> int:
    """The C ``fa_fwd``: device pointers as ints, returns the status code."""
    return load_library().fa_fwd(q, k, v, o, lse or None, B, H, N, d, scale, int(bool(causal)),
                                 stream or None)


def fa_fwd_noalloc(q: int, k: int, v: int, o: int, lse: int | None, B: int, H: int, N: int, d: int,
                   scale: float, causal: bool, stream: int | None) -> int:
    """The C ``fa_fwd_noalloc``: ``fa_fwd`` for callers that cannot let the
    library allocate device memory (its scratch is a fixed array inside the
    library). Calls whose kernels overlap on the GPU share that scratch and
    must not be issued. Returns the status code."""
    return load_library().fa_fwd_noalloc(q, k, v, o, lse or None, B, H, N, d, scale, int(bool(causal)),
                                         stream or None)


def fa_fwd_varlen(q: int, k: int, v: int, o: int, lse: int | None, cu_q: int, cu_k: int, B: int, H: int,
                  total_q: int, total_k: int, max_seqlen_q: int, d: int, scale: float, causal: bool,
                  stream: int | None) -> int:
    """The C ``fa_fwd_varlen``: device pointers as ints, returns the status code."""
    return load_library().fa_fwd_varlen(q, k, v, o, lse or None, cu_q, cu_k, B, H, total_q, total_k,
                                        max_seqlen_q, d, scale, int(bool(causal)), stream or None)


def fa_varlen_num_splits(B: int, H: int, total_k: int, max_seqlen_q: int, sm_count: int) -> int:
    """The C ``fa_varlen_num_splits`` (host only): work items per unit's key
    range that ``fa_fwd_varlen`` uses for these sizes, or a negative status."""
    return load_library().fa_varlen_num_splits(B, H, total_k, max_seqlen_q, sm_count)


def fa_strerror(status: int) -> str:
    return load_library().fa_strerror(status).decode()


def fa_device_status(stream: int | None = None) -> tuple[int, int]:
    """Synchronises ``stream``, reads and clears the device status word."""
    bits = ctypes.c_uint(0)
    rc = load_library().fa_device_status(stream or None, ctypes.byref(bits))
    return rc, bits.value


def fa_set_wait_limit_ns(ns: int) -> None:
    load_library().fa_set_wait_limit_ns(ns)


def fa_abi_version() -> int:
    return load_library().fa_abi_version()


def fa_selftest_wait_timeout(limit_ns: int, stream: int | None = None) -> int:
    """The C ``fa_selftest_wait_timeout``: one warp waits on a barrier that
    nothing completes until ``limit_ns`` passes, then records the timeout in
    the device status word. Returns the launch status."""
    return load_library().fa_selftest_wait_timeout(stream or None, limit_ns)


def fa_selftest_exp2(x: int, y_approx: int, y_exp2f: int, n: int, stream: int | None = None) -> int:
    """The C ``fa_selftest_exp2``: 2^x on the device by the softmax's
    ex2.approx.ftz.f32 and by CUDA's exp2f, for n fp32 arguments (device
    pointers as ints). Returns the status code."""
    return load_library().fa_selftest_exp2(x, y_approx, y_exp2f, n, stream or None)


# fa_selftest_ex2_rate: threads per block and chains per thread
EX2_RATE_THREADS = 1024
EX2_RATE_CHAINS = 8


def fa_selftest_ex2_rate(cycles: int, sink: int, blocks: int, iters: int, stream: int | None = None) -> int:
    """The C ``fa_selftest_ex2_rate``: ``blocks`` blocks (one per SM) each
    run EX2_RATE_THREADS x EX2_RATE_CHAINS chains of ``iters`` dependent
    ex2.approx; ``cycles`` (device int64 [blocks]) receives each block's span
    in SM clocks, ``sink`` (device fp32 [blocks * EX2_RATE_THREADS]) the
    chains' last values. Returns the status code."""
    return load_library().fa_selftest_ex2_rate(cycles, sink, blocks, iters, stream or None)


def fa_decode_paged(q: int, cache: FaPagedCache, block_table: int, seq_lens: int, o: int, lse: int | None, B: int,
                    Hq: int, table_width: int, table_stride: int, scale: float, workspace: int, workspace_bytes: int,
                    stream: int | None) -> int:
    """The C ``fa_decode_paged``: device pointers as ints, returns the status code."""
    return load_library().fa_decode_paged(q, ctypes.byref(cache), block_table, seq_lens, o, lse or None, B, Hq,
                                          table_width, table_stride, scale, workspace or None, workspace_bytes,
                                          stream or None)


def fa_decode_paged_workspace(B: int, Hq: int, Hkv: int, d: int, cache_type: int, page_size: int, table_width: int,
                              sm_count: int) -> int:
    """The C ``fa_decode_paged_workspace`` (host only): workspace bytes of
    ``fa_decode_paged`` for these sizes, or a negative status."""
    return load_library().fa_decode_paged_workspace(B, Hq, Hkv, d, cache_type, page_size, table_width, sm_count)


def fa_rotary(x: int, y: int, positions: int, inv_freq: int | None, B: int, H: int, N: int, d: int, x_strides,
              y_strides, position_stride: int, rotary_dim: int, interleaved: bool, inverse: bool, factor: float,
              stream: int | None) -> int:
    """The C ``fa_rotary``: device pointers as ints, ``x_strides`` and
    ``y_strides`` of three elements (b, h, n). Returns the status code."""
    three = ctypes.c_longlong * 3
    return load_library().fa_rotary(x, y, positions, inv_freq or None, B, H, N, d, three(*x_strides),
                                    three(*y_strides), position_stride, rotary_dim, int(bool(interleaved)),
                                    int(bool(inverse)), factor, stream or None)


def fa_cache_append(q: int, k: int, v: int, q_stride: int, k_stride: int, v_stride: int, positions: int, slots: int,
                    inv_freq: int | None, cache: FaPagedCache, q_out: int, k_out: int | None, q_out_stride: int,
                    k_out_stride: int, T: int, Hq: int, rotary_dim: int, interleaved: bool, factor: float,
                    stream: int | None) -> int:
    """The C ``fa_cache_append``: device pointers as ints, returns the status code."""
    return load_library().fa_cache_append(q, k, v, q_stride, k_stride, v_stride, positions, slots, inv_freq or None,
                                          ctypes.byref(cache), q_out, k_out or None, q_out_stride, k_out_stride, T,
                                          Hq, rotary_dim, int(bool(interleaved)), factor, stream or None)


def fa_page_maps(context_lens: int, new_lens: int, block_table: int, unused_blocks: int, slots: int, positions: int,
                 cu_seqlens: int, seq_lens: int, counts: int, B: int, table_width: int, table_stride: int,
                 num_unused: int, page_size: int, T: int, stream: int | None) -> int:
    """The C ``fa_page_maps``: device pointers as ints, returns the status code."""
    return load_library().fa_page_maps(context_lens, new_lens, block_table, unused_blocks, slots, positions,
                                       cu_seqlens, seq_lens, counts, B, table_width, table_stride, num_unused,
                                       page_size, T, stream or None)


def _current_stream_handle(torch, device) -> int:
    """The raw cudaStream_t of the current stream on `device` (without
    building a Stream object when torch offers the raw handle)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(device.index if device.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


def attention_forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
                      return_lse: bool = True, stream=None):
    """O (bf16) and LSE (fp32) for bf16 CUDA tensors q, k, v of shape [B, H, N, d].

    ``out`` / ``lse`` may be given to reuse buffers. Runs on ``stream`` (a
    torch.cuda.Stream) or the current stream.
    """
    import torch
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k, v must be bf16")
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must all be [B, H, N, d]")
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    sp = stream.cuda_stream if stream is not None else _current_stream_handle(torch, q.device)
    rc = (_lib or load_library()).fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                         lse.data_ptr() if lse is not None else None, B, H, N, d, float(scale),
                                         1 if causal else 0, sp or None)
    if rc != FA_OK:
        raise FaError(rc)
    return (out, lse) if return_lse else out


def attention_forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, causal: bool = False,
                             scale: float | None = None, out=None, lse=None, return_lse: bool = True,
                             stream=None):
    """O [total_q, H, d] (bf16) and LSE [H, total_q] (fp32) for a batch of
    sequences of different lengths: q [total_q, H, d], k and v [total_k, H, d]
    (bf16, CUDA, contiguous), int32 CUDA offsets ``cu_seqlens_q`` /
    ``cu_seqlens_k`` of B + 1 entries. Under ``causal`` each sequence's last
    query is aligned with its last key."""
    import torch
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k, v must be bf16")
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or q.shape[1:] != k.shape[1:]:
        raise ValueError("q must be [total_q, H, d] and k, v [total_k, H, d]")
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens_q.dim() != 1 or cu_seqlens_k.shape != cu_seqlens_q.shape or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both hold B + 1 offsets")
    for t in (q, k, v, cu_seqlens_q, cu_seqlens_k):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all inputs must be contiguous CUDA tensors")
    total_q, H, d = q.shape
    total_k = k.shape[0]
    B = cu_seqlens_q.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    sp = stream.cuda_stream if stream is not None else _current_stream_handle(torch, q.device)
    rc = fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                       lse.data_ptr() if lse is not None else None, cu_seqlens_q.data_ptr(),
                       cu_seqlens_k.data_ptr(), B, H, total_q, total_k, int(max_seqlen_q), d, float(scale),
                       causal, sp)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_varlen")
    return (out, lse) if return_lse else out


def head_shards(num_heads_total: int, world: int) -> list[tuple[int, int]]:
    """Contiguous ranges (start, count) of the flattened B*H head axis for
    ``world`` ranks, in rank order, sizes differing by at most one (the first
    ``num_heads_total % world`` ranks take one more). Heads are independent
    (each head's O and LSE depend only on its own Q, K, V), so a rank that
    holds its range's Q, K, V computes its O and LSE alone: the head-sharded
    multi-GPU forward needs no exchange between ranks."""
    if num_heads_total < 0 or world < 1:
        raise ValueError("need num_heads_total >= 0 and world >= 1")
    base, extra = divmod(num_heads_total, world)
    out, start = [], 0
    for r in range(world):
        n = base + (1 if r < extra else 0)
        out.append((start, n))
        start += n
    return out


def attention_forward_heads(q, k, v, head_start: int, head_count: int, causal: bool = False,
                            scale: float | None = None, out=None, lse=None, stream=None):
    """fa_fwd on heads [head_start, head_start + head_count) of the flattened
    B*H axis of contiguous bf16 CUDA tensors [B, H, N, d]: the C call gets
    pointers into q, k, v (and into ``out`` / ``lse``, allocated whole when
    not given), nothing is copied, and the other heads of ``out`` and ``lse``
    are left as they were. Returns (out, lse) for the whole [B, H, N, d] /
    [B, H, N] shape. Each rank of a head-sharded job calls this on the range
    ``head_shards(B*H, world)[rank]`` of tensors in its own device memory."""
    import torch
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k, v must be bf16")
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must all be [B, H, N, d]")
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    B, H, N, d = q.shape
    if head_start < 0 or head_count < 0 or head_start + head_count > B * H:
        raise ValueError("head range outside [0, B*H)")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if head_count == 0:
        return out, lse
    eo, el = N * d * q.element_size(), N * 4   # bytes per head of q/k/v/out and of lse
    sp = stream.cuda_stream if stream is not None else _current_stream_handle(torch, q.device)
    rc = fa_fwd(q.data_ptr() + head_start * eo, k.data_ptr() + head_start * eo, v.data_ptr() + head_start * eo,
                out.data_ptr() + head_start * eo, lse.data_ptr() + head_start * el, 1, head_count, N, d,
                float(scale), causal, sp)
    if rc != FA_OK:
        raise FaError(rc)
    return out, lse


# ---- serving from a paged cache, rotary positions ---------------------------


# struct fa_paged_cache as bytes (laid out as FaPagedCache), which a call takes in
# a tenth of the time that building the ctypes structure does
_pack_cache = struct.Struct("PPPPqqqqqqiiiii4x").pack


def _launch(torch, fn, args, device, stream, made, what):
    """``fn(*args, stream handle)`` with CUDA device number ``device`` current.
    Tensors that were made for the call belong to the current stream's part of
    the allocator; when another ``stream`` uses them it is told so, so that none
    is handed out again while that stream's kernels may still run."""
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        handle = raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    else:
        handle = stream.cuda_stream
        for t in made:
            t.record_stream(stream)
    if device == torch.cuda.current_device():
        rc = fn(*args, handle or None)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle or None)
    if rc != FA_OK:
        raise FaError(rc, what)


def _elsewhere(device, tensors):
    """Raises for the tensors (of those that are not None) that are not on CUDA
    device number ``device``; -1 is the CPU."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("all tensors must be on the same CUDA device")


def _pack_paged_cache(torch, device, k_cache, v_cache, k_scale, v_scale):
    """(struct fa_paged_cache as bytes, its type) of caches indexed [block,
    token, head, d]."""
    t = k_cache.dtype
    if t is torch.bfloat16:
        kind = CACHE_BF16
    elif t is torch.float8_e4m3fn:
        kind = CACHE_E4M3
    else:
        raise TypeError("k_cache and v_cache must both be bf16 or both float8_e4m3fn")
    if v_cache.dtype is not t:
        raise TypeError("k_cache and v_cache must both be bf16 or both float8_e4m3fn")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both be [num_blocks, page_size, heads, d]")
    kb, kt, kh, kd = k_cache.stride()
    vb, vt, vh, vd = v_cache.stride()
    if kd != 1 or vd != 1:
        raise ValueError("the d values of a cache row must be contiguous")
    if k_cache.get_device() != device or v_cache.get_device() != device:
        _elsewhere(device, (k_cache, v_cache))
    scales = [0, 0]
    for i, x in enumerate((k_scale, v_scale)):
        if x is not None:
            if x.dtype is not torch.float32 or x.shape != (shape[2],) or not x.is_contiguous():
                raise ValueError("k_scale and v_scale must be contiguous fp32 tensors of one value per key head")
            _elsewhere(device, (x,))
            scales[i] = x.data_ptr()
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), *scales, kb, kt, kh, vb, vt, vh, kind, *shape), kind


@functools.lru_cache(maxsize=256)
def _decode_workspace_bytes(B, Hq, Hkv, d, cache_type, page_size, table_width, device_index):
    import torch
    sms = torch.cuda.get_device_properties(device_index).multi_processor_count
    n = fa_decode_paged_workspace(B, Hq, Hkv, d, cache_type, page_size, table_width, sms)
    if n < 0:
        raise FaError(n, "fa_decode_paged_workspace")
    return n


def attention_decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None, k_scale=None,
                           v_scale=None, out=None, lse=None, return_lse: bool = True, workspace=None, stream=None):
    """O [B, Hq, d] (bf16) and LSE [B, Hq] (fp32) of one new token per request
    over its pages: q [B, Hq, d] (bf16), ``k_cache`` / ``v_cache`` indexed
    [num_blocks, page_size, heads, d] (bf16 or float8_e4m3fn, any order in
    memory with d innermost: a permuted or sliced view will do), int32
    ``block_table`` [B, width] and ``seq_lens`` [B] (keys of each request, the
    new token's among them). Hq is a multiple of heads. A value of the cache is
    its element times ``k_scale`` / ``v_scale`` [heads] (fp32), where given.
    A request without keys gets O = 0, LSE = -inf.

    ``workspace`` (uint8, at least ``fa_decode_paged_workspace`` bytes) may be
    given to keep allocation out of the call; calls that may overlap in time
    need one each."""
    import torch
    if q.dtype is not torch.bfloat16:
        raise TypeError("q must be bf16")
    if block_table.dtype is not torch.int32 or seq_lens.dtype is not torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [B, Hq, d], block_table [B, width] and seq_lens [B]")
    device = q.get_device()
    if device < 0:
        raise ValueError("all inputs must be CUDA tensors")
    B, Hq, d = q.shape
    rows, width = block_table.shape
    if rows != B or seq_lens.shape != (B,):
        raise ValueError("q must be [B, Hq, d], block_table [B, width] and seq_lens [B]")
    row_stride, step = block_table.stride()
    if (step != 1 and width > 1) or not q.is_contiguous() or not seq_lens.is_contiguous():
        raise ValueError("q, seq_lens and the rows of block_table must be contiguous")
    _elsewhere(device, (block_table, seq_lens, out, lse, workspace))
    cache, kind = _pack_paged_cache(torch, device, k_cache, v_cache, k_scale, v_scale)
    _, page, heads, cache_d = k_cache.shape
    if cache_d != d:
        raise ValueError("q and the caches must have the same d")
    made = ()
    if out is None:
        out = torch.empty_like(q)
        made = (out,)
    elif out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor of q's shape")
    if lse is None:
        if return_lse:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
            made += (lse,)
    elif lse.dtype is not torch.float32 or lse.shape != (B, Hq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, Hq]")
    if workspace is None:
        room = _decode_workspace_bytes(B, Hq, heads, d, kind, page, width, device)
        workspace = torch.empty(room, dtype=torch.uint8, device=q.device)
        made += (workspace,)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    else:
        room = workspace.numel()
    _launch(torch, (_lib or load_library()).fa_decode_paged,
            (q.data_ptr(), cache, block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
             lse.data_ptr() if lse is not None else None, B, Hq, width, row_stride, 1.0 / math.sqrt(d) if scale is None
             else scale, workspace.data_ptr(), room), device, stream, made, "fa_decode_paged")
    return (out, lse) if return_lse else out


def rotary_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None, device=None):
    """(inv_freq, factor) for ``rotary`` and ``cache_append``: fp64 [rotary_dim
    / 2] frequencies base^(-2i / rotary_dim) on ``device`` and the factor of cos
    and sin, laid out once per model. ``scaling`` stretches them for contexts
    longer than the trained one, by ``{"type": ...}``:

    * ``"linear"``, ``factor``: every frequency divided by factor.
    * ``"ntk"``, ``factor``: base raised by factor^(r / (r - 2)), so that the
      slowest frequency is divided by factor and the fastest is kept.
    * ``"bands"``, ``factor``, ``original`` (trained context), ``low`` = 1,
      ``high`` = 4: frequencies that turn less than ``low`` times over the
      trained context are divided by factor, those that turn more than
      ``high`` times are kept, linear in the number of turns between.
    * ``"yarn"``, ``factor``, ``original``, ``low`` = 1, ``high`` = 32,
      ``attention_factor`` = 0.1 ln(factor) + 1: the same, linear in the
      frequency's index between, and cos and sin times attention_factor.
    """
    import torch
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and >= 0")
    if not (math.isfinite(base) and base > 0):
        raise ValueError("base must be finite and > 0")
    r = rotary_dim
    index = torch.arange(0, r, 2, dtype=torch.float64)
    freq, out_factor = float(base) ** (-index / r) if r else index, 1.0
    if scaling is not None:
        kind, factor = scaling.get("type"), float(scaling.get("factor", 1.0))
        if not (math.isfinite(factor) and factor > 0):
            raise ValueError("scaling factor must be finite and > 0")
        if kind == "linear":
            freq = freq / factor
        elif kind == "ntk":
            if r > 2:
                freq = (base * factor ** (r / (r - 2))) ** (-index / r)
        elif kind in ("bands", "yarn"):
            original = float(scaling["original"])
            low, high = float(scaling.get("low", 1.0)), float(scaling.get("high", 4.0 if kind == "bands" else 32.0))
            if not (original > 0 and 0 < low < high):
                raise ValueError("scaling needs original > 0 and 0 < low < high")
            if kind == "bands":
                keep = ((original * freq / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
            else:
                # the (fractional) indexes whose frequencies turn `high` and `low` times over the trained context
                i_high, i_low = (r * math.log(original / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low))
                first, last = max(math.floor(i_high), 0), min(math.ceil(i_low), r - 1)
                keep = 1 - ((index / 2 - first) / max(last - first, 1e-3)).clamp(0, 1)
                out_factor = float(scaling.get("attention_factor", 0.1 * math.log(factor) + 1 if factor > 1 else 1.0))
            freq = freq * keep + freq / factor * (1 - keep)
        else:
            raise ValueError(f"unknown rotary scaling {kind!r}")
    return (freq.to(device) if device is not None else freq), out_factor


def _frequencies(torch, device, inv_freq):
    """(rotary_dim, pointer) of the frequencies; none: (0, None)."""
    if inv_freq is None:
        return 0, None
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous fp64 tensor [rotary_dim / 2]")
    if inv_freq.get_device() != device:
        _elsewhere(device, (inv_freq,))
    return 2 * inv_freq.shape[0], inv_freq.data_ptr() or None


_three = struct.Struct("qqq").pack  # strides, as the C call reads them


def rotary(x, positions, inv_freq, interleaved: bool = False, inverse: bool = False, factor: float = 1.0, out=None,
           stream=None):
    """Rotary positions of x (bf16, CUDA): [B, H, N, d] with int32 ``positions``
    [N] or [B, N], or token-major [T, H, d] with positions [T]. Any strides with
    d contiguous. ``inv_freq`` (fp64 [rotary_dim / 2]) and ``factor`` are those of
    ``rotary_inv_freq``; pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1) when
    ``interleaved``. ``inverse`` turns back by the same angles (times factor):
    the gradient with respect to x. ``out`` may be x. Not differentiable by
    itself: ``torch.ops.fa91.rotary`` is."""
    import torch
    if x.dtype is not torch.bfloat16:
        raise TypeError("x must be bf16")
    if positions.dtype is not torch.int32:
        raise TypeError("positions must be int32")
    device = x.get_device()
    if device < 0:
        raise ValueError("x must be a CUDA tensor")
    shape, pos_stride = x.shape, 0
    if len(shape) == 4:
        B, H, N, d = shape
        sb, sh, sn, sd = x.stride()
        if positions.dim() == 2 and positions.shape == (B, N):
            pos_stride, step = positions.stride()
        elif positions.shape == (N,):
            step, = positions.stride()
        else:
            raise ValueError("positions must be [N] or [B, N]")
    elif len(shape) == 3:
        (N, H, d), B, sb = shape, 1, 0
        sn, sh, sd = x.stride()
        if positions.shape != (N,):
            raise ValueError("positions must be [T]")
        step, = positions.stride()
    else:
        raise ValueError("x must be [B, H, N, d] or [T, H, d]")
    if sd != 1 or (step != 1 and N > 1):
        raise ValueError("d of x and the rows of positions must be contiguous")
    _elsewhere(device, (positions, out))
    r, freq = _frequencies(torch, device, inv_freq)
    made = ()
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
        made = (out,)
    elif out.dtype is not torch.bfloat16 or out.shape != shape or out.stride(-1) != 1:
        raise ValueError("out must be a bf16 tensor of x's shape with d contiguous")
    if len(shape) == 4:
        tb, th, tn, _ = out.stride()
    else:
        (tn, th, _), tb = out.stride(), 0
    _launch(torch, (_lib or load_library()).fa_rotary,
            (x.data_ptr(), out.data_ptr(), positions.data_ptr(), freq, B, H, N, d, _three(sb, sh, sn),
             _three(tb, th, tn), pos_stride, r, 1 if interleaved else 0, 1 if inverse else 0, factor), device, stream,
            made, "fa_rotary")
    return out


def cache_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved: bool = False,
                 factor: float = 1.0, k_scale=None, v_scale=None, q_out=None, k_out=None, stream=None):
    """One step's tokens into a paged cache: q [T, Hq, d] and k [T, heads, d]
    (bf16, CUDA) turned by their rotary positions (``inv_freq`` None: not
    turned), k and v [T, heads, d] written to their ``slots`` (int32 [T]; slot s
    is token s % page_size of block s // page_size) of ``k_cache`` /
    ``v_cache`` [num_blocks, page_size, heads, d], q returned turned (in
    ``q_out`` where given; it may be q). ``k_out`` [T, heads, d] also receives
    the turned k (for a prompt's own attention; it may be k). A token with a
    negative slot is padding: nothing of it is written anywhere. q, k and v may
    be slices of one projection's output. float8_e4m3fn caches hold value /
    scale, with ``k_scale`` / ``v_scale`` fp32 [heads] (None: 1)."""
    import torch
    bf16 = torch.bfloat16
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16:
        raise TypeError("q, k, v must be bf16")
    if positions.dtype is not torch.int32 or slots.dtype is not torch.int32:
        raise TypeError("positions and slots must be int32")
    device = q.get_device()
    if device < 0:
        raise ValueError("all inputs must be CUDA tensors")
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape:
        raise ValueError("q must be [T, Hq, d] and k, v [T, heads, d]")
    T, Hq, d = q.shape
    Tk, heads, dk = k.shape
    if Tk != T or dk != d or k_cache.shape[2:] != (heads, d):
        raise ValueError("q, k, v and the caches do not fit together")
    if positions.shape != (T,) or slots.shape != (T,) or not positions.is_contiguous() or not slots.is_contiguous():
        raise ValueError("positions and slots must be contiguous [T]")
    _elsewhere(device, (k, v, positions, slots, q_out, k_out))
    cache, _ = _pack_paged_cache(torch, device, k_cache, v_cache, k_scale, v_scale)
    r, freq = _frequencies(torch, device, inv_freq)
    made = ()
    if q_out is None:
        q_out = torch.empty((T, Hq, d), dtype=bf16, device=q.device)
        made = (q_out,)
    elif q_out.dtype is not bf16 or q_out.shape != q.shape:
        raise ValueError("q_out must be bf16 and of q's shape")
    if k_out is not None and (k_out.dtype is not bf16 or k_out.shape != k.shape):
        raise ValueError("k_out must be bf16 and of k's shape")
    strides = []
    for t, h in ((q, Hq), (k, heads), (v, heads), (q_out, Hq), (k_out, heads)):
        if t is None:
            strides.append(0)
            continue
        row, head, step = t.stride()
        if step != 1 or (head != d and h > 1):
            raise ValueError("the heads of a token of q, k, v, q_out and k_out must be contiguous")
        strides.append(row)
    _launch(torch, (_lib or load_library()).fa_cache_append,
            (q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides[:3], positions.data_ptr(), slots.data_ptr(), freq,
             cache, q_out.data_ptr(), k_out.data_ptr() if k_out is not None else None, *strides[3:], T, Hq, r,
             1 if interleaved else 0, factor), device, stream, made, "fa_cache_append")
    return q_out


class PageMaps(typing.NamedTuple):
    """What ``page_maps`` gives for a step (int32 CUDA tensors)."""
    slots: "torch.Tensor"        # [T] where each new token goes (cache_append)
    positions: "torch.Tensor"    # [T] its position in its request
    cu_seqlens: "torch.Tensor"   # [B + 1] offsets of the requests' new tokens (attention_forward_varlen)
    seq_lens: "torch.Tensor"     # [B] keys of each request after the step (attention_decode_paged)
    counts: "torch.Tensor"       # [4] pages taken, pages missing, new tokens, requests past the table's width


def page_maps(context_lens, new_lens, block_table, unused_blocks, page_size: int, num_tokens: int,
              out: PageMaps | None = None, stream=None) -> PageMaps:
    """Block tables and slot maps of one step, made on the GPU from request
    lengths (int32 CUDA tensors): request b holds ``context_lens``[b] tokens and
    gets ``new_lens``[b] more. ``block_table`` [B, width] is completed in place
    with the blocks that the new tokens need, taken from ``unused_blocks`` in
    order (the caller then drops the first ``counts[0]``); ``num_tokens`` is the
    length of the token maps, which may be more than the step's tokens (the
    rest are padding: slot -1). See ``fa_page_maps`` in include/fa.h."""
    import torch
    i32 = torch.int32
    if (context_lens.dtype is not i32 or new_lens.dtype is not i32 or block_table.dtype is not i32 or
            unused_blocks.dtype is not i32):
        raise TypeError("context_lens, new_lens, block_table and unused_blocks must be int32")
    device = block_table.get_device()
    if device < 0:
        raise ValueError("all inputs must be CUDA tensors")
    if block_table.dim() != 2 or unused_blocks.dim() != 1:
        raise ValueError("block_table must be [B, width] and unused_blocks one list")
    B, width = block_table.shape
    row_stride, step = block_table.stride()
    if context_lens.shape != (B,) or new_lens.shape != (B,):
        raise ValueError("context_lens and new_lens must be [B]")
    if ((step != 1 and width > 1) or not context_lens.is_contiguous() or not new_lens.is_contiguous() or
            not unused_blocks.is_contiguous()):
        raise ValueError("the rows of block_table, the lengths and unused_blocks must be contiguous")
    _elsewhere(device, (context_lens, new_lens, unused_blocks))
    T = int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must be >= 0")
    made = ()
    if out is None:
        whole = torch.empty(2 * T + 2 * B + 5, dtype=i32, device=block_table.device)
        out = PageMaps(*whole.split_with_sizes((T, T, B + 1, B, 4)))
        made = (whole,)
    else:
        for t, n in zip(out, (T, T, B + 1, B, 4)):
            if t.dtype is not i32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != device:
                raise ValueError("out must be int32 tensors [T], [T], [B + 1], [B] and [4] on the same device")
    slots, positions, cu_seqlens, seq_lens, counts = out
    _launch(torch, (_lib or load_library()).fa_page_maps,
            (context_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), unused_blocks.data_ptr() or None,
             slots.data_ptr() or None, positions.data_ptr() or None, cu_seqlens.data_ptr(), seq_lens.data_ptr(),
             counts.data_ptr(), B, width, row_stride, unused_blocks.shape[0], page_size, T), device, stream, made,
            "fa_page_maps")
    return out

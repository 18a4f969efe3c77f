"""Python binding of libfa.so, the GB300 (sm_103a) exact-attention forward.

The C entry points (``include/fa.h``) are exposed under the same names and
take raw device pointers (ints), exactly like the C ABI. ``attention_forward``
is a convenience wrapper for torch tensors: it checks dtypes and layout,
allocates the outputs with torch and calls ``fa_fwd`` on the current stream.
Every step of the computation runs in the CUDA library; if the library is
missing this module raises instead of computing anything elsewhere. The
serving functions (paged cache, rotary positions) do the same through the
binding's native half, ``lib/_fa_bind-torch<version>.so``: their kernels are
often shorter than what the checks and the call cost in Python.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import typing

from .build import BIND_PATH, LIB_PATH

__all__ = ["FaError", "load_library", "fa_fwd", "fa_fwd_noalloc", "fa_strerror", "fa_device_status",
           "fa_set_wait_limit_ns", "fa_abi_version", "fa_selftest_wait_timeout", "fa_fwd_varlen",
           "fa_varlen_num_splits", "fa_selftest_exp2", "fa_selftest_ex2_rate", "EX2_RATE_THREADS",
           "EX2_RATE_CHAINS", "attention_forward", "attention_forward_varlen",
           "head_shards", "attention_forward_heads", "EXPORTED_SYMBOLS", "CACHE_BF16", "CACHE_E4M3",
           "FaPagedCache", "fa_decode_paged", "fa_decode_paged_workspace", "fa_rotary", "fa_cache_append",
           "fa_page_maps", "attention_decode_paged", "rotary", "rotary_inv_freq", "cache_append", "page_maps",
           "PageMaps", "load_binding"]

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
    torch.cuda.Stream) or the current stream. On another stream than the current
    one the caller keeps the tensors, results included, until the work is done
    (``Tensor.record_stream``): their memory belongs to the current stream.
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
    query is aligned with its last key. ``stream`` as in ``attention_forward``."""
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
    ``head_shards(B*H, world)[rank]`` of tensors in its own device memory.
    ``stream`` as in ``attention_forward``."""
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


_bind = None


def load_binding():
    """The binding's native half (``lib/_fa_bind-torch<version>.so``, built with
    libfa.so): the checks, allocations and C calls of the functions below."""
    global _bind
    if _bind is None:
        import torch  # noqa: F401  (its libraries, which the module is linked to)
        if not os.path.exists(BIND_PATH):
            raise FileNotFoundError(
                f"{BIND_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
        load_library()
        spec = importlib.util.spec_from_file_location("_fa_bind", BIND_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.setup(FaError, PageMaps)
        _bind = module
    return _bind


def _on_stream(stream, device, fn, *args):
    """fn(*args) with ``stream`` as the current one. What the call allocates then
    belongs to that stream's part of the allocator (memory that the current
    stream's earlier work may still use is not written), and results are not
    handed out again there while the current stream may still read them, nor the
    memory of tensors given (temporaries) while ``stream`` may still use it."""
    import torch
    if stream.device != device:
        raise ValueError("stream must be one of the tensors' device")
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        r = fn(*args)
    for a in args:
        for t in a if isinstance(a, tuple) else (a,):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    for t in r if isinstance(r, tuple) else (r,):
        t.record_stream(current)
    return r


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
    need one each.

    Runs on ``stream`` (a torch.cuda.Stream) or the current stream, as the
    functions below do. The work is ordered on that stream alone; the memory of
    tensors that are dropped meanwhile is not handed out again before it is done."""
    decode = (_bind or load_binding()).decode
    if stream is None:
        return decode(q, k_cache, v_cache, block_table, seq_lens, scale, k_scale, v_scale, out, lse, return_lse,
                      workspace)
    return _on_stream(stream, q.device, decode, q, k_cache, v_cache, block_table, seq_lens, scale, k_scale, v_scale,
                      out, lse, return_lse, workspace)


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


def rotary(x, positions, inv_freq, interleaved: bool = False, inverse: bool = False, factor: float = 1.0, out=None,
           stream=None):
    """Rotary positions of x (bf16, CUDA): [B, H, N, d] with int32 ``positions``
    [N] or [B, N], or token-major [T, H, d] with positions [T]. Any strides that
    are multiples of 8, d contiguous, at a 16-byte boundary. ``inv_freq`` (fp64 [rotary_dim / 2]) and ``factor`` are those of
    ``rotary_inv_freq``; pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1) when
    ``interleaved``. ``inverse`` turns back by the same angles (times factor):
    the gradient with respect to x. ``out`` may be x. Not differentiable by
    itself: ``torch.ops.fa91.rotary`` is."""
    turn = (_bind or load_binding()).rotary
    if stream is None:
        return turn(x, positions, inv_freq, interleaved, inverse, factor, out)
    return _on_stream(stream, x.device, turn, x, positions, inv_freq, interleaved, inverse, factor, out)


def cache_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved: bool = False,
                 factor: float = 1.0, k_scale=None, v_scale=None, q_out=None, k_out=None, stream=None):
    """One step's tokens into a paged cache: q [T, Hq, d] and k [T, heads, d]
    (bf16, CUDA) turned by their rotary positions (``inv_freq`` None: not
    turned), k and v [T, heads, d] written to their ``slots`` (int32 [T]; slot s
    is token s % page_size of block s // page_size) of ``k_cache`` /
    ``v_cache`` [num_blocks, page_size, heads, d], q returned turned (in
    ``q_out`` where given; it may be q). ``k_out`` [T, heads, d] also receives
    the turned k (for a prompt's own attention; it may be k). A token with a
    negative slot is padding: nothing of it is written anywhere (its row of a
    q_out that the call makes is not initialised). q, k and v may be slices of
    one projection's output. float8_e4m3fn caches hold value / scale, with
    ``k_scale`` / ``v_scale`` fp32 [heads] (None: 1)."""
    append = (_bind or load_binding()).append
    if stream is None:
        return append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved, factor, k_scale, v_scale,
                      q_out, k_out)
    return _on_stream(stream, q.device, append, q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved,
                      factor, k_scale, v_scale, q_out, k_out)


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
    maps = (_bind or load_binding()).maps
    if stream is None:
        return maps(context_lens, new_lens, block_table, unused_blocks, page_size, num_tokens, out)
    return _on_stream(stream, block_table.device, maps, context_lens, new_lens, block_table, unused_blocks, page_size,
                      num_tokens, out)

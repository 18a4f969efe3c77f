"""PyTorch custom operators over the C ABI.

``torch.ops.fa91.attention_forward(q, k, v, causal, scale)`` returns
``(O, LSE)`` for bf16 CUDA tensors ``[B, H, N, d]``, computed by ``fa_fwd``
(the same kernels as :func:`exact_attention_91_gb300.attention_forward`).
``torch.ops.fa91.attention_forward_varlen(q, k, v, cu_seqlens_q,
cu_seqlens_k, max_seqlen_q, causal, scale)`` returns ``(O [total_q, H, d],
LSE [H, total_q])`` for packed sequences, computed by ``fa_fwd_varlen``. The
attention operators are forward-only: the attention backward pass is not part
of this library. ``torch.ops.fa91.rotary`` (rotary positions) is
differentiable. ``attention_decode_paged``, ``cache_append`` and ``page_maps``
serve from a paged cache, as the functions of the same names do; the last two
change their caches or block table in place. (``cache_append`` here has no
``k_out``: a prompt's own attention takes its keys from ``torch.ops.fa91.rotary``.)
The fake (meta) implementations
give output shapes and dtypes without a GPU, so the operators can be traced.
"""
from __future__ import annotations

import torch

from . import (PageMaps, attention_decode_paged, attention_forward, attention_forward_varlen, cache_append, page_maps,
               rotary)


@torch.library.custom_op("fa91::attention_forward", mutates_args=())
def attention_forward_op(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                         scale: float | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    o, lse = attention_forward(q, k, v, causal=causal, scale=scale, return_lse=True)
    return o, lse


@attention_forward_op.register_fake
def _attention_forward_fake(q, k, v, causal=False, scale=None):
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must all be [B, H, N, d]")
    B, H, N, _ = q.shape
    return torch.empty_like(q), q.new_empty((B, H, N), dtype=torch.float32)


@torch.library.custom_op("fa91::attention_forward_varlen", mutates_args=())
def attention_forward_varlen_op(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                                cu_seqlens_k: torch.Tensor, max_seqlen_q: int, causal: bool = False,
                                scale: float | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    o, lse = attention_forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal=causal,
                                      scale=scale, return_lse=True)
    return o, lse


@attention_forward_varlen_op.register_fake
def _attention_forward_varlen_fake(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal=False, scale=None):
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or q.shape[1:] != k.shape[1:]:
        raise ValueError("q must be [total_q, H, d] and k, v [total_k, H, d]")
    total_q, H, _ = q.shape
    return torch.empty_like(q), q.new_empty((H, total_q), dtype=torch.float32)


@torch.library.custom_op("fa91::attention_decode_paged", mutates_args=())
def attention_decode_paged_op(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_table: torch.Tensor, seq_lens: torch.Tensor, scale: float | None = None,
                              k_scale: torch.Tensor | None = None,
                              v_scale: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    o, lse = attention_decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale=scale, k_scale=k_scale,
                                    v_scale=v_scale)
    return o, lse


@attention_decode_paged_op.register_fake
def _attention_decode_paged_fake(q, k_cache, v_cache, block_table, seq_lens, scale=None, k_scale=None, v_scale=None):
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("q must be [B, Hq, d] and the caches [num_blocks, page_size, heads, d]")
    B, Hq, _ = q.shape
    return torch.empty_like(q), q.new_empty((B, Hq), dtype=torch.float32)


@torch.library.custom_op("fa91::rotary", mutates_args=())
def rotary_op(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor | None, interleaved: bool = False,
              inverse: bool = False, factor: float = 1.0) -> torch.Tensor:
    return rotary(x, positions, inv_freq, interleaved=interleaved, inverse=inverse, factor=factor)


@rotary_op.register_fake
def _rotary_fake(x, positions, inv_freq, interleaved=False, inverse=False, factor=1.0):
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B, H, N, d] or [T, H, d]")
    return x.new_empty(x.shape)


def _rotary_setup(ctx, inputs, output):
    _, positions, inv_freq, ctx.interleaved, ctx.inverse, ctx.factor = inputs
    ctx.save_for_backward(positions, inv_freq)


def _rotary_backward(ctx, grad):
    # the map is linear: its gradient is the transposed map, the turn back by the same angles
    positions, inv_freq = ctx.saved_tensors
    if grad.stride(-1) != 1 or grad.storage_offset() % 8 or any(s % 8 for s in grad.stride()[:-1]):
        grad = grad.clone(memory_format=torch.contiguous_format)  # (a reduction's broadcast gradient, a slice)
    dx = torch.ops.fa91.rotary(grad, positions, inv_freq, ctx.interleaved, not ctx.inverse, ctx.factor)
    return dx, None, None, None, None, None


rotary_op.register_autograd(_rotary_backward, setup_context=_rotary_setup)


@torch.library.custom_op("fa91::cache_append", mutates_args=("k_cache", "v_cache"))
def cache_append_op(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                    inv_freq: torch.Tensor | None, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    interleaved: bool = False, factor: float = 1.0, k_scale: torch.Tensor | None = None,
                    v_scale: torch.Tensor | None = None) -> torch.Tensor:
    return cache_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved=interleaved, factor=factor,
                        k_scale=k_scale, v_scale=v_scale)


@cache_append_op.register_fake
def _cache_append_fake(q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved=False, factor=1.0,
                       k_scale=None, v_scale=None):
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape:
        raise ValueError("q must be [T, Hq, d] and k, v [T, heads, d]")
    return q.new_empty(q.shape)


@torch.library.custom_op("fa91::page_maps", mutates_args=("block_table",))
def page_maps_op(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                 unused_blocks: torch.Tensor, page_size: int,
                 num_tokens: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    B = block_table.shape[0]
    out = PageMaps(*(torch.empty(n, dtype=torch.int32, device=block_table.device)
                     for n in (num_tokens, num_tokens, B + 1, B, 4)))
    return tuple(page_maps(context_lens, new_lens, block_table, unused_blocks, page_size, num_tokens, out=out))


@page_maps_op.register_fake
def _page_maps_fake(context_lens, new_lens, block_table, unused_blocks, page_size, num_tokens):
    B = block_table.shape[0]
    return tuple(block_table.new_empty(n) for n in (num_tokens, num_tokens, B + 1, B, 4))

"""What moves tokens into and out of the paged cache around the decode step:
append_kv_norm (QK norms, rotary embedding and the paged write in one pass)
and evict_kv (cut sequences back to a budget by accumulated attention weight).

All compute runs in libfd.
"""
from __future__ import annotations

import torch

from . import _lib


def _pool_sizes(entry, k_pages, block_table):
    """(num_pages, page_size, Hkv, D), max_blocks of the pool and its table."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError(f"{entry}: k_pages must be a tensor [num_pages, page_size, Hkv, D]")
    if k_pages.dtype not in (torch.float16, torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"{entry}: k_pages must be float16, bfloat16 or float8_e4m3fn, got {k_pages.dtype}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError(f"{entry}: block_table must be a tensor [B, max_blocks]")
    return k_pages.shape, block_table.shape[1]


def append_kv_norm(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, q_weight=None, k_weight=None, eps=1e-6,
                   rotary_cos=None, rotary_sin=None, interleaved=False, positions=None, new_lens=None, k_scale=None,
                   v_scale=None, q_out=None, status=None, stream=None):
    """Norm and rotate q [B, T, Hq, D] and k_new [B, T, Hkv, D] head by head,
    write k_new and v_new at cache slots seq_lens[b] + i, and return the
    queries (q_out, allocated when not given; q itself for in place).

    Without T ([B, heads, D]) each sequence takes one token.  q may be None
    (K and V only).  q_weight / k_weight [D]: RMS norm with that weight (None:
    no norm); rotary_cos / rotary_sin fp32 [max_pos, rotary_dim / 2] (None: no
    rotation); positions int32 [B]: rotary position of each sequence's first
    token (None: seq_lens, right while nothing was evicted); new_lens int32
    [B]: tokens of each sequence in this call (None: T; rows of q_out beyond
    are not written).  seq_lens is not advanced."""
    if stream is None and (fast := _lib.fast()):
        done = fast.append_kv_norm(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, q_weight, k_weight, eps,
                                   rotary_cos, rotary_sin, interleaved, positions, new_lens, k_scale, v_scale, q_out,
                                   status)
        if done is not None:
            return done[0]
    if not isinstance(k_new, torch.Tensor) or k_new.dim() not in (3, 4):
        raise ValueError("append_kv_norm: k_new must be a tensor [B, T, Hkv, D] or [B, Hkv, D]")
    if q is not None and (not isinstance(q, torch.Tensor) or q.dim() != k_new.dim()):
        raise ValueError("append_kv_norm: q must have k_new's dimensions")
    if k_new.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"append_kv_norm: k_new must be float16 or bfloat16, got {k_new.dtype}")
    Hkv, D = k_new.shape[-2:]
    Hq = Hkv if q is None else q.shape[-2]
    (num_pages, page_size, _, _), max_blocks = _pool_sizes("append_kv_norm", k_pages, block_table)
    prob = _lib.make_problem(k_new.shape[0], Hq, Hkv, D, page_size, max_blocks, num_pages, k_new.dtype, k_pages.dtype)
    if q is not None and q_out is None:
        q_out = _lib.empty_on(q.shape, q.dtype, q.device, stream)
    _lib.fd_append_kv_norm(prob, q, k_new, v_new, q_out, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens,
                           q_weight, k_weight, eps, rotary_cos, rotary_sin, interleaved, positions, new_lens, status,
                           stream)
    return q_out


def evict_kv(k_pages, v_pages, block_table, seq_lens, weights, budget, sinks=0, recent=0, dst_table=None,
             weights_out=None, k_scale=None, v_scale=None, status=None, stream=None):
    """Cut every sequence longer than budget back to budget tokens: the first
    sinks, the last recent and, per KV head, the others with the largest
    weights [B, Hkv, N] stay, moved up in their order.

    In place (dst_table None) or into the pages of dst_table, which
    block_table must not name.  E4M3 codes that move to a page with another
    scale are rescaled, rounded and saturated at 448 each time they do.
    weights_out (weights for in place; None: not kept) receives the kept
    weights.  Returns (new_lens int32 [B], kept int32 [B, Hkv, budget], the old
    indices, -1 past a row's new length)."""
    if stream is None and (fast := _lib.fast()):
        done = fast.evict_kv(k_pages, v_pages, block_table, seq_lens, weights, budget, sinks, recent, dst_table,
                             weights_out, k_scale, v_scale, status)
        if done is not None:
            return done
    (num_pages, page_size, Hkv, D), max_blocks = _pool_sizes("evict_kv", k_pages, block_table)
    B = block_table.shape[0]
    act = torch.bfloat16 if k_pages.dtype == torch.float8_e4m3fn else k_pages.dtype  # the op has no activations
    prob = _lib.make_problem(B, Hkv, Hkv, D, page_size, max_blocks, num_pages, act, k_pages.dtype)
    if int(budget) < 1:
        raise ValueError("evict_kv: budget must be at least 1")
    if budget > page_size * max_blocks:  # as the call itself would, but before kept is allocated
        raise _lib.FdError(_lib.FD_ERR_INVALID_ARG, f"evict_kv: budget {budget} of a table for {page_size * max_blocks}")
    new_lens = _lib.empty_on((B,), torch.int32, k_pages.device, stream)
    kept = _lib.empty_on((B, Hkv, int(budget)), torch.int32, k_pages.device, stream)
    _lib.fd_evict_kv(prob, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights, weights_out, budget,
                     sinks, recent, new_lens, kept, dst_table, status, stream)
    return new_lens, kept

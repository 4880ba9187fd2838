"""Attention over states that many query rows share: cross attention to an
encoder's cached states (CrossDecoder) and decode of sequences behind shared
prefixes (PrefixDecoder).

All compute runs in libfd.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib


class _Planned:
    """Workspace and device status word of a plan (self.plan)."""

    def _reserve(self, device):
        self.device = torch.device(device)
        self.workspace = torch.zeros(max(256, int(self.plan.workspace_bytes)), dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        if self.device.type == "cuda" and not torch.cuda.is_current_stream_capturing():
            # finish the fills before a call on another stream runs
            torch.cuda.current_stream(self.device).synchronize()

    def check(self):
        """Synchronise the decoder's device and raise FdError if the device
        reported an error."""
        if self.device.type == "cuda":
            torch.cuda.synchronize(self.device)
        word = int(self.status.item())
        if word:
            self.status.zero_()
            self.workspace.zero_()
            if self.device.type == "cuda":
                # finish the clears before a call on another stream runs
                torch.cuda.synchronize(self.device)
            raise _lib.FdError(_lib.fd_status_from_device(word), "device status")


class CrossDecoder(_Planned):
    """Cross attention of decoder tokens to an encoder's states in the paged
    pools: a plan with its workspace and status word, used like PagedDecoder
    (lengths may change within the plan's capacity; calls on one decoder must
    not overlap on the GPU).

    problem.B counts KV rows (one per encoded input); beams sequences in a row
    read each of them, tokens query tokens each.  Over bf16 pools the softmax
    weights of many query rows have one bf16 part; weight_parts=2 gives them the
    two of PagedDecoder."""

    def __init__(self, problem, kv_lens_host, tokens=1, beams=1, device="cuda", **plan_opts):
        self.problem = problem
        self.plan = _lib.fd_plan_cross(problem, kv_lens_host, tokens=tokens, beams=beams, **plan_opts)
        self._reserve(device)

    @classmethod
    def for_pools(cls, q, k_pages, v_pages, block_table, kv_lens_host, beams=1, **plan_opts):
        """q [B, Hq, D] or [B, T, Hq, D] for T query tokens per sequence;
        block_table [B / beams, max_blocks].  max_kv_len reserves room for
        longer inputs."""
        if q.dim() not in (3, 4):
            raise ValueError("q must be [B, Hq, D] or [B, T, Hq, D]")
        num_pages, page_size, Hkv, D = k_pages.shape
        if D != q.shape[-1]:
            raise ValueError("head dimension of q and the pools differ")
        if beams < 1 or q.shape[0] != block_table.shape[0] * beams:
            raise ValueError("q must hold beams sequences for every row of block_table")
        prob = _lib.make_problem(block_table.shape[0], q.shape[-2], Hkv, D, page_size, block_table.shape[1], num_pages,
                                 q.dtype, k_pages.dtype)
        return cls(prob, kv_lens_host, tokens=q.shape[1] if q.dim() == 4 else 1, beams=beams, device=q.device, **plan_opts)

    def __call__(self, q, k_pages, v_pages, block_table, kv_lens, q_lens=None, k_scale=None, v_scale=None, out=None,
                 lse=None, want_lse=True, stream=None):
        """q's tokens may lie at a stride (a slice of a fused projection);
        q_lens int32 [B]: tokens of each sequence in this call (None: all T;
        rows of out and lse beyond are not written).  Returns (out, lse)."""
        if stream is None and (fast := _lib.fast()):
            done = fast.cross(ctypes.addressof(self.plan), q, k_pages, v_pages, block_table, kv_lens, q_lens, k_scale, v_scale,
                              out, lse, want_lse, self.workspace, self.status)
            if done is not None:
                return done
        if not isinstance(q, torch.Tensor):
            raise ValueError("CrossDecoder: q must be a tensor")
        if out is None:
            out = _lib.empty_on(q.shape, q.dtype, self.device, stream)
        if lse is None and want_lse:
            lse = _lib.empty_on(q.shape[:-1], torch.float32, self.device, stream)
        _lib.fd_cross_paged(self.plan, q, k_pages, v_pages, k_scale, v_scale, block_table, kv_lens, out, lse,
                            self.workspace, q_lens, self.status, stream)
        return out, lse


class PrefixDecoder(_Planned):
    """Decode of a batch whose sequences share prefixes, several groups of
    them: every prefix is attended once for all of its sequences, each
    sequence's own tokens as in PagedDecoder, and the two are joined.

    prefix_of: for each sequence the index of its prefix, or -1 for none, in
    any order.  regroup() changes it without a new plan.  weight_parts=1 rounds
    the softmax weights of bf16 prefixes to one bf16, which is faster."""

    def __init__(self, problem, seq_lens_host, prefix_max_blocks, prefix_lens_host, prefix_of, device="cuda",
                 **plan_opts):
        self.problem = problem
        self.prefixes = len(prefix_lens_host)
        members, offsets = self._grouped(prefix_of)
        self.plan = _lib.fd_plan_prefix(problem, seq_lens_host, prefix_max_blocks, prefix_lens_host, offsets, **plan_opts)
        self._reserve(device)
        self.members, self.offsets = members.to(self.device), offsets.to(self.device)

    @classmethod
    def for_pools(cls, q, k_pages, v_pages, prefix_table, prefix_lens_host, prefix_of, block_table, seq_lens_host,
                  **plan_opts):
        """q [B, Hq, D], or [B, q_len, Hq, D] for q_len causal query tokens per
        sequence (its last q_len own tokens); prefix_table [P, blocks] and
        prefix_lens_host of the prefixes, block_table [B, blocks] and
        seq_lens_host of the sequences' own tokens."""
        if q.dim() == 4:
            plan_opts.setdefault("q_len", q.shape[1])
        num_pages, page_size, Hkv, D = k_pages.shape
        if D != q.shape[-1]:
            raise ValueError("head dimension of q and the pools differ")
        prob = _lib.make_problem(q.shape[0], q.shape[-2], Hkv, D, page_size, block_table.shape[1], num_pages, q.dtype,
                                 k_pages.dtype)
        return cls(prob, seq_lens_host, prefix_table.shape[1], prefix_lens_host, prefix_of, device=q.device, **plan_opts)

    def _grouped(self, prefix_of):
        """(members, offsets) of fd_decode_paged_prefix, on the host."""
        of = _lib._host_i32("PrefixDecoder", "prefix_of", prefix_of, self.problem.B)
        if of.numel() and (int(of.min()) < -1 or int(of.max()) >= self.prefixes):
            raise ValueError(f"PrefixDecoder: prefix_of must be -1 to {self.prefixes - 1}")
        key = torch.where(of < 0, self.prefixes, of)
        counts = torch.bincount(key, minlength=self.prefixes + 1)[:self.prefixes]
        offsets = torch.zeros(self.prefixes + 1, dtype=torch.int32)
        offsets[1:] = counts.cumsum(0)
        return key.sort(stable=True).indices.to(torch.int32), offsets

    def regroup(self, prefix_of):
        """Take another prefix_of from the next call on (written on the
        current stream, also for a captured graph's replays)."""
        members, offsets = self._grouped(prefix_of)
        self.members.copy_(members)
        self.offsets.copy_(offsets)

    def __call__(self, q, k_pages, v_pages, prefix_table, prefix_lens, block_table, seq_lens, k_scale=None, v_scale=None,
                 out=None, lse=None, want_lse=True, stream=None):
        """prefix_lens int32 [P], seq_lens int32 [B] (own tokens, after this
        step's were appended).  Returns (out, lse)."""
        if stream is None and (fast := _lib.fast()):
            done = fast.decode_prefix(ctypes.addressof(self.plan), q, k_pages, v_pages, prefix_table, prefix_lens, self.members,
                                      self.offsets, block_table, seq_lens, k_scale, v_scale, out, lse, want_lse,
                                      self.workspace, self.status)
            if done is not None:
                return done
        if not isinstance(q, torch.Tensor):
            raise ValueError("PrefixDecoder: q must be a tensor")
        if out is None:
            out = _lib.empty_on(q.shape, q.dtype, self.device, stream)
        if lse is None and want_lse:
            lse = _lib.empty_on(q.shape[:-1], torch.float32, self.device, stream)
        _lib.fd_decode_paged_prefix(self.plan, q, k_pages, v_pages, k_scale, v_scale, prefix_table, prefix_lens,
                                    self.members, self.offsets, block_table, seq_lens, out, lse, self.workspace,
                                    self.status, stream)
        return out, lse

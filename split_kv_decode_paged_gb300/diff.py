"""Differential attention over the paged cache: the difference of two softmax
maps, with learned weights, and the norm of each head.

A head has two queries of width d (q's halves), the cache two keys of width d
(the halves of a K row) and one value of width D = 2 d:

    out_h = softmax(q1 k1^T / sqrt(d)) V - lam_h softmax(q2 k2^T / sqrt(d)) V
    out_h = out_h * rsqrt(mean(out_h^2) + eps) * norm_weight * out_scale

lam_h is the model's exp(lq1 . lk1) - exp(lq2 . lk2) + lam_init, a constant of
the weights; out_scale its 1 - lam_init.  All compute runs in libfd.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib


class DiffDecoder:
    """A differential-attention plan with its workspace and status word; used
    like PagedDecoder (the same plan options, capacity and overlap rules).
    problem.Hq counts differential heads, problem.D is both maps' width."""

    def __init__(self, problem, seq_lens_host, device="cuda", **plan_opts):
        self.problem = problem
        self.plan = _lib.fd_plan_diff(problem, seq_lens_host, **plan_opts)
        self.device = torch.device(device)
        self.workspace = torch.zeros(max(256, int(self.plan.workspace_bytes)), dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    @classmethod
    def for_pools(cls, q, k_pages, v_pages, block_table, seq_lens_host, out_dtype=None, **plan_opts):
        """q [B, Hq, D], or [B, q_len, Hq, D] for q_len causal query tokens
        per sequence (the last q_len cached tokens of each)."""
        if q.dim() == 4:
            plan_opts.setdefault("q_len", q.shape[1])
        num_pages, page_size, Hkv, D = k_pages.shape
        if D != q.shape[-1]:
            raise ValueError("head dimension of q and the pools differ")
        prob = _lib.make_problem(q.shape[0], q.shape[-2], Hkv, D, page_size, block_table.shape[1], num_pages, q.dtype,
                                 k_pages.dtype, out_dtype)
        return cls(prob, seq_lens_host, device=q.device, **plan_opts)

    def __call__(self, q, k_pages, v_pages, block_table, seq_lens, lam, norm_weight=None, eps=1e-5, out_scale=1.0,
                 k_scale=None, v_scale=None, out=None, lse=None, want_lse=True, stream=None):
        """lam fp32 [Hq]; norm_weight [D] in q's type or fp32 (None: no norm).
        Returns (out like q, lse fp32 [..., Hq, 2] of both maps or None)."""
        if stream is None and (fast := _lib.fast()):
            done = fast.decode_diff(ctypes.addressof(self.plan), q, k_pages, v_pages, block_table, seq_lens, lam,
                                    norm_weight, eps, out_scale, k_scale, v_scale, out, lse, want_lse, self.workspace,
                                    self.status)
            if done is not None:
                return done
        p, plan = self.problem, self.plan
        lead = (p.B,) if plan.q_len <= 1 else (p.B, plan.q_len)
        if out is None:
            out = _lib.empty_on(lead + (p.Hq, p.D), _lib.FD_TO_TORCH[p.out_dtype], self.device, stream)
        if lse is None and want_lse:
            lse = _lib.empty_on(lead + (p.Hq, 2), torch.float32, self.device, stream)
        _lib.fd_decode_paged_diff(plan, q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, lam, out, lse,
                                  self.workspace, norm_weight, eps, out_scale, self.status, stream)
        return out, lse

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
                torch.cuda.synchronize(self.device)
            raise _lib.FdError(_lib.fd_status_from_device(word), "device status")

"""Refusals of append_kv_norm, decode_weights, evict_kv and differential
attention: bad arguments raise before anything is launched, so these run
without a GPU (at the C ABI with addresses that are never dereferenced, in
the binding with host tensors, whose placement is checked last)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUP, SMALL = _lib.FD_ERR_INVALID_ARG, _lib.FD_ERR_UNSUPPORTED, _lib.FD_ERR_WORKSPACE_TOO_SMALL
A = 1 << 20  # an address that is never dereferenced
REF = ctypes.byref


def prob(**kw):
    base = dict(B=2, Hq=8, Hkv=2, D=128, page_size=16, max_blocks_per_seq=8, num_pages=64, q_dtype=torch.bfloat16,
                kv_dtype=torch.bfloat16)
    base.update(kw)
    return _lib.make_problem(**base)


# ------------------------------------------------------------------ C ABI
def norm_args(**kw):
    n = _lib.FdNormAppend(tokens=2, q=A, k_new=A, v_new=A, q_out=A, q_stride=1024, k_stride=256, v_stride=256,
                          q_out_stride=1024, q_weight=A, k_weight=A, weight_dtype=_lib.FD_BF16, eps=1e-6, rotary_cos=A,
                          rotary_sin=A, rotary_dim=128, max_pos=64, interleaved=0)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def call_append(lib, n, p=None, k=A, v=A, ks=None, vs=None, bt=A, sl=A):
    return lib.fd_append_kv_norm(REF(p or prob()), None if n is None else REF(n), k, v, ks, vs, bt, sl, None, None)


@pytest.mark.parametrize("kw", [dict(tokens=0), dict(k_new=None), dict(v_new=None), dict(q=None), dict(q_out=None),
                                dict(q=A + 8), dict(k_new=A + 2), dict(v_new=A + 4), dict(q_out=A + 8),
                                dict(q_stride=1020), dict(q_stride=1016), dict(k_stride=0), dict(v_stride=-256),
                                dict(q_out_stride=512), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")),
                                dict(eps=float("nan")), dict(q_weight=A + 1), dict(weight_dtype=_lib.FD_F16),
                                dict(weight_dtype=_lib.FD_E4M3), dict(weight_dtype=_lib.FD_F32, k_weight=A + 2),
                                dict(rotary_sin=None), dict(rotary_cos=None), dict(rotary_dim=0), dict(rotary_dim=3),
                                dict(rotary_dim=130), dict(max_pos=0), dict(rotary_cos=A + 2), dict(positions=A + 2),
                                dict(new_lens=A + 1)])
def test_append_rejects_bad_arguments(fdlib, kw):
    assert call_append(fdlib, norm_args(**kw)) == BAD


def test_append_rejects_bad_pools_and_problems(fdlib):
    n = norm_args()
    assert call_append(fdlib, None) == BAD
    for kw in (dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 4), dict(bt=None), dict(sl=None), dict(bt=A + 2),
               dict(ks=A, vs=A)):
        assert call_append(fdlib, n, **kw) == BAD, kw
    p8 = prob(kv_dtype=torch.float8_e4m3fn)
    assert call_append(fdlib, n, p=p8) == BAD
    assert call_append(fdlib, n, p=p8, ks=A, vs=A + 2) == BAD
    assert call_append(fdlib, n, p=prob(D=96)) == UNSUP
    assert call_append(fdlib, n, p=prob(page_size=24)) == BAD
    assert call_append(fdlib, norm_args(q_out_stride=2048)) == BAD  # q itself at another stride
    assert call_append(fdlib, norm_args(q_stride=1 << 40, q_out_stride=1 << 40), p=prob(Hq=1 << 21)) == UNSUP
    # a grid beyond what a launch can have
    big = prob(B=8192)
    assert call_append(fdlib, norm_args(tokens=0x7fffffff), p=big) == UNSUP


def weights_call(lib, plan, ws=None, wws=None, **kw):
    a = dict(q=A, k=A, v=A, ks=None, vs=None, bt=A, sl=A, out=A, lse=None, w=None, wo=A, stride=100, w_ws=A)
    a.update(kw)
    n = _lib.fd_decode_weights_workspace(plan) if wws is None else wws
    return lib.fd_decode_paged_weights(REF(plan), a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["sl"], a["out"],
                                       a["lse"], a["w"], a["wo"], a["stride"], A,
                                       plan.workspace_bytes if ws is None else ws, a["w_ws"], n, None, None)


def test_weights_rejects_bad_arguments(fdlib):
    plan = _lib.fd_plan(prob(), [100, 50], num_sms=152)
    for kw in (dict(q=None), dict(k=A + 8), dict(out=None), dict(wo=None), dict(stride=0), dict(wo=A + 2),
               dict(w=A + 2), dict(w_ws=None), dict(w_ws=A + 128), dict(w=A + 4, wo=A), dict(ks=A, vs=A)):
        assert weights_call(fdlib, plan, **kw) == BAD, kw
    # disjoint and equal arrays pass that check (2 x 2 x 100 floats) and stop at the next one
    for w in (A, A + 1600, A - 1600):
        assert weights_call(fdlib, plan, w=w, q=None) == BAD
    assert weights_call(fdlib, plan, w=A + 1596) == BAD
    assert weights_call(fdlib, plan, wws=_lib.fd_decode_weights_workspace(plan) - 1) == SMALL
    assert weights_call(fdlib, plan, ws=plan.workspace_bytes - 1) == SMALL
    shared = _lib.fd_plan(prob(), [100], num_sms=152, shared_kv=1)
    assert fdlib.fd_decode_weights_workspace(REF(shared), REF(ctypes.c_size_t())) == UNSUP
    diff = _lib.fd_plan_diff(prob(), [100, 50], num_sms=152)
    assert fdlib.fd_decode_weights_workspace(REF(diff), REF(ctypes.c_size_t())) == BAD
    assert fdlib.fd_decode_weights_workspace(None, REF(ctypes.c_size_t())) == BAD
    wide = _lib.fd_plan(prob(Hq=8 * 1024, Hkv=1, D=64), [100, 50], num_sms=152)
    assert fdlib.fd_decode_weights_workspace(REF(wide), REF(ctypes.c_size_t())) == UNSUP


def test_weights_workspace_covers_the_capacity(fdlib):
    """One score for every token of capacity and query row, and the lse."""
    plan = _lib.fd_plan(prob(), [100, 50], num_sms=152, max_seq_len=128)
    assert _lib.fd_decode_weights_workspace(plan) >= 2 * 8 * 4 * (plan.capacity_tokens + 1)
    plan = _lib.fd_plan(prob(), [100, 50], num_sms=152, q_len=3)
    assert _lib.fd_decode_weights_workspace(plan) >= 2 * 3 * 8 * 4 * (plan.capacity_tokens + 1)


def evict_call(lib, p=None, **kw):
    a = dict(k=A, v=A, ks=None, vs=None, bt=A, sl=A, w=A, wo=A, stride=100, budget=20, sinks=2, recent=5, dst=None, n=A + 64,
             kept=A)
    a.update(kw)
    return lib.fd_evict_kv(REF(p or prob()), a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["sl"], a["w"], a["wo"], a["stride"],
                           a["budget"], a["sinks"], a["recent"], a["dst"], a["n"], a["kept"], None, None)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=A + 8), dict(bt=None), dict(sl=None), dict(w=None), dict(w=A + 2),
                                dict(wo=A + 4), dict(stride=0), dict(budget=0), dict(budget=-1), dict(sinks=-1),
                                dict(recent=-1), dict(sinks=21), dict(sinks=10, recent=11), dict(budget=129, sinks=0),
                                dict(n=None), dict(kept=None), dict(n=A), dict(dst=A + 2), dict(ks=A, vs=A),
                                dict(sinks=2147483647, recent=2147483647)])
def test_evict_rejects_bad_arguments(fdlib, kw):
    assert evict_call(fdlib, **kw) == BAD


def test_evict_rejects_bad_problems(fdlib):
    assert evict_call(fdlib, p=prob(kv_dtype=torch.float8_e4m3fn)) == BAD
    assert evict_call(fdlib, p=prob(D=96)) == UNSUP


def diff_call(lib, plan, ws=None, **kw):
    a = dict(q=A, k=A, v=A, ks=None, vs=None, bt=A, sl=A, lam=A, nw=A, wt=_lib.FD_BF16, eps=1e-5, out=A, lse=None, work=A)
    a.update(kw)
    return lib.fd_decode_paged_diff(REF(plan), a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["sl"], a["lam"], a["nw"],
                                    a["wt"], a["eps"], 1.0, a["out"], a["lse"], a["work"],
                                    plan.workspace_bytes if ws is None else ws, None, None)


def test_diff_rejects_bad_arguments(fdlib):
    plan = _lib.fd_plan_diff(prob(), [100, 50], num_sms=152)
    for kw in (dict(q=None), dict(q=A + 8), dict(k=None), dict(k=A + 8), dict(bt=None), dict(sl=A + 1), dict(lam=None),
               dict(lam=A + 2), dict(nw=A + 1), dict(wt=_lib.FD_F16), dict(wt=_lib.FD_E4M3), dict(eps=0.0),
               dict(eps=float("nan")), dict(out=None), dict(out=A + 8), dict(lse=A + 2), dict(work=None),
               dict(work=A + 128), dict(ks=A, vs=A)):
        assert diff_call(fdlib, plan, **kw) == BAD, kw
    assert diff_call(fdlib, plan, ws=plan.workspace_bytes - 1) == SMALL
    assert diff_call(fdlib, _lib.fd_plan(prob(), [100, 50], num_sms=152)) == BAD  # a plain plan
    # and a differential plan is not for the plain call
    assert fdlib.fd_decode_paged(REF(plan), A, A, A, None, None, A, A, A, None, A, plan.workspace_bytes, None, None) == BAD


def test_diff_plan_is_the_plan_of_the_doubled_heads(fdlib):
    plan = _lib.fd_plan_diff(prob(), [100, 50], num_sms=152)
    two = _lib.fd_plan(prob(Hq=16), [100, 50], num_sms=152)
    a, b = plan.as_dict(), two.as_dict()
    assert a == b
    assert fdlib.fd_plan_diff(None, None, None, None) == BAD
    for kw, code in ((dict(Hq=6, Hkv=4), BAD), (dict(D=96), UNSUP), (dict(D=32), UNSUP)):
        with pytest.raises(_lib.FdError) as e:
            _lib.fd_plan_diff(prob(**kw), [10, 10], num_sms=152)
        assert e.value.code == code
    with pytest.raises(_lib.FdError) as e:
        _lib.fd_plan_diff(prob(), [10], num_sms=152, shared_kv=1)
    assert e.value.code == UNSUP


def test_norm_append_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    py = _lib.FdNormAppend
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "fd_api.h"', 'int main(void) {',
             'printf("size %zu\\n", sizeof(fd_norm_append));']
    lines += [f'printf("{f} %zu\\n", offsetof(fd_norm_append, {f}));' for f, _ in py._fields_] + ["return 0; }"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, value = line.split()
        assert int(value) == (ctypes.sizeof(py) if name == "size" else getattr(py, name).offset), name


# ---------------------------------------------------------------- binding
B, T, HQ, HKV, D, PS, MB, NP = 2, 3, 8, 2, 128, 16, 4, 12
BF = torch.bfloat16


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def append_kw(**kw):
    a = dict(q=z(B, T, HQ, D), k_new=z(B, T, HKV, D), v_new=z(B, T, HKV, D), k_pages=z(NP, PS, HKV, D),
             v_pages=z(NP, PS, HKV, D), block_table=z(B, MB, dtype=torch.int32), seq_lens=z(B, dtype=torch.int32),
             q_weight=z(D), k_weight=z(D), rotary_cos=z(9, 64, dtype=torch.float32),
             rotary_sin=z(9, 64, dtype=torch.float32), q_out=z(B, T, HQ, D))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,msg", [
    (dict(k_new=None), "k_new"), (dict(k_new=z(B, HKV * D)), "k_new"), (dict(q=z(B, HQ, D)), "q must"),
    (dict(q=z(B, T, HQ, D, dtype=torch.float16)), "q must have dtype"), (dict(v_new=z(B, T, HKV + 1, D)), "v_new.*shape"),
    (dict(k_new=z(B, 0, HKV, D), q=z(B, 0, HQ, D)), "at least one token"),
    (dict(v_new=z(B, T, D, HKV).transpose(2, 3)), "v_new.*contiguous heads"),
    (dict(v_new=z(B, 2 * T, HKV, D)[:, ::2][:, :T].contiguous().expand(B, T, HKV, D)[:, :, :1].expand(B, T, HKV, D)),
     "v_new.*contiguous heads"),
    (dict(k_new=z(T, B, HKV, D).transpose(0, 1)), "k_new.*one stride"),
    (dict(v_new=z(1, 1, HKV, D).expand(B, T, HKV, D)), "v_new.*(one|token) stride"),
    (dict(v_new=z(B, T, HKV * D + 4)[..., :HKV * D].unflatten(-1, (HKV, D))), "v_new.*multiple of 8"),
    (dict(q_weight=z(64)), "q_weight.*shape"), (dict(k_weight=z(D, dtype=torch.float32)), "k_weight.*dtype"),
    (dict(rotary_sin=None), "rotary_sin is required"), (dict(rotary_cos=None), "rotary_cos is required"),
    (dict(rotary_cos=z(9, dtype=torch.float32)), "2-D"), (dict(positions=z(B, dtype=torch.int64)), "positions.*dtype"),
    (dict(new_lens=z(B + 1, dtype=torch.int32)), "new_lens.*shape"), (dict(k_scale=z(1)), "k_scale must be None"),
    (dict(v_pages=z(NP, PS, HKV, 64)), "v_pages.*shape"), (dict(block_table=z(B, MB)), "block_table.*dtype"),
    (dict(k_new=z(B, T, HKV, D, dtype=torch.float32)), "k_new must be float16 or bfloat16"),
    (dict(k_pages=None), "k_pages must be a tensor"), (dict(k_pages=z(NP, PS, HKV, D, dtype=torch.float32)), "k_pages must be float16"),
    (dict(block_table=None), "block_table must be a tensor"), (dict(q=None), "q_out must be None"), (dict(q_out=z(B, T, HQ, D, dtype=torch.float32)), "q_out.*dtype"),
    (dict(), "must be a CUDA tensor"),
])
def test_append_binding_refusals(fdlib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        fd.append_kv_norm(**append_kw(**kw))


@pytest.mark.parametrize("kw,msg", [
    (dict(budget=0), "budget"), (dict(k_pages=None), "k_pages"), (dict(block_table=z(B)), "block_table must be a tensor"), (dict(weights=z(B, HKV, 50)), "weights.*dtype"),
    (dict(weights=z(B, HKV + 1, 50, dtype=torch.float32)), "weights.*shape"),
    (dict(weights_out=z(B, HKV, 51, dtype=torch.float32)), "weights_out.*shape"),
    (dict(dst_table=z(B, MB + 1, dtype=torch.int32)), "dst_table.*shape"), (dict(seq_lens=z(B)), "seq_lens.*dtype"),
    (dict(k_scale=z(1)), "k_scale must be None"), (dict(), "must be a CUDA tensor"),
])
def test_evict_binding_refusals(fdlib, kw, msg):
    a = dict(k_pages=z(NP, PS, HKV, D), v_pages=z(NP, PS, HKV, D), block_table=z(B, MB, dtype=torch.int32),
             seq_lens=z(B, dtype=torch.int32), weights=z(B, HKV, 50, dtype=torch.float32), budget=20)
    a.update(kw)
    with pytest.raises(ValueError, match=msg):
        fd.evict_kv(**a)


def test_decode_weights_binding_refusals(fdlib):
    p = prob(max_blocks_per_seq=MB, num_pages=NP)
    args = (z(B, HQ, D), z(NP, PS, HKV, D), z(NP, PS, HKV, D), z(B, MB, dtype=torch.int32), z(B, dtype=torch.int32))
    plain = fd.PagedDecoder(p, [40, 50], device="cpu", num_sms=152)
    w = z(B, HKV, 64, dtype=torch.float32)
    with pytest.raises(ValueError, match="track_weights"):
        plain.decode_weights(*args, w)
    dec = fd.PagedDecoder(p, [40, 50], device="cpu", num_sms=152, track_weights=True)
    for bad, msg in ((None, "weights_out is required"), (z(B, HKV, 64), "weights_out.*dtype"),
                     (z(B, HKV + 1, 64, dtype=torch.float32), "weights_out.*shape"),
                     (z(HKV, 64, dtype=torch.float32), "weights_out.*shape"), (w, "CUDA")):
        with pytest.raises(ValueError, match=msg):
            dec.decode_weights(*args, bad)
    with pytest.raises(ValueError, match="weights must have shape"):
        dec.decode_weights(*args, z(B, HKV, 63, dtype=torch.float32), weights_out=w)


def test_diff_binding_refusals(fdlib):
    p = prob(max_blocks_per_seq=MB, num_pages=NP)
    dec = fd.DiffDecoder(p, [40, 50], device="cpu", num_sms=152)
    base = dict(q=z(B, HQ, D), k_pages=z(NP, PS, HKV, D), v_pages=z(NP, PS, HKV, D),
                block_table=z(B, MB, dtype=torch.int32), seq_lens=z(B, dtype=torch.int32),
                lam=z(HQ, dtype=torch.float32))
    for kw, msg in ((dict(lam=z(HQ)), "lam.*dtype"), (dict(lam=z(2 * HQ, dtype=torch.float32)), "lam.*shape"),
                    (dict(q=z(B, 2 * HQ, D)), "q must have shape"), (dict(norm_weight=z(D, dtype=torch.float16)), "norm_weight"),
                    (dict(norm_weight=z(64)), "norm_weight.*shape"), (dict(lse=z(B, HQ, dtype=torch.float32)), "lse.*shape"),
                    (dict(out=z(B, HQ, D, dtype=torch.float32)), "out.*dtype"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=msg):
            dec(**{**base, **kw})
    with pytest.raises(ValueError, match="fd_plan_diff"):
        plan = _lib.fd_plan(p, [40, 50], num_sms=152)
        _lib.fd_decode_paged_diff(plan, base["q"], base["k_pages"], base["v_pages"], None, None, base["block_table"],
                                  base["seq_lens"], base["lam"], z(B, HQ, D), None, z(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="head dimension"):
        fd.DiffDecoder.for_pools(z(B, HQ, 64), base["k_pages"], base["v_pages"], base["block_table"], [4, 4])

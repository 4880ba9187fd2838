"""The bits in which the softmax weights enter P.V where an output goes by the
lse itself: differential attention over maps that resemble each other, where a
rounding of the weights would be scaled up with what is left of them."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests import cache_ref as R
from tests.test_gpu_weights import setup

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def moved(p, v, err):
    """How far sum p v may be off: every weight by twice its score's error, by
    2^-21 (a pair of f16 halves holds 22 bits) and by 2^-25 of the largest one
    (f16's floor; the largest is at least 1 before the division), the sums and
    factors in fp32 by 2^-18."""
    return (2.0 ** -21 + 2 * err + 2.0 ** -18) * torch.einsum("hgn,nhd->hgd", p, v.abs()) + 2.0 ** -25 * v.abs().sum(0)[:, None]


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("norm,out_dtype", [(False, torch.float32), (True, torch.float32), (True, None)])
@pytest.mark.parametrize("D,Hq,Hkv,ps,q_len", [(128, 8, 2, 16, 1), (64, 8, 2, 64, 1), (128, 16, 1, 32, 1), (128, 8, 2, 64, 4)])
def test_difference_of_similar_maps_over_e4m3(fdlib, act, norm, out_dtype, D, Hq, Hkv, ps, q_len):
    lens = [4, 5, 9, 40, 300]
    q, kp, vp, ks, vs, bt = setup("e4m3", act, lens, Hq, Hkv, D, ps, q_len, seed=D + Hq)
    gen = torch.Generator().manual_seed(5)
    w = D // 2
    kp.view(torch.uint8)[..., w:] = kp.view(torch.uint8)[..., :w]
    q[..., w:] = (q[..., :w].float() * (1 + 0.03 * torch.randn(q[..., w:].shape, generator=gen))).to(q.dtype)
    nw = 1 + 0.3 * torch.randn(D, generator=gen) if norm else None
    dec = fd.DiffDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, out_dtype=out_dtype)
    out, _ = dec(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                 torch.ones(Hq).cuda(), norm_weight=nw.cuda() if norm else None, eps=1e-5, k_scale=ks.cuda(), v_scale=vs.cuda())
    torch.cuda.synchronize()
    dec.check()
    od = DT[act] if out_dtype is None else out_dtype
    out = out.cpu().double().reshape(len(lens), q_len, Hq, D)
    kd, vd = R.values(kp, ks), R.values(vp, vs)
    qd = q.float().double().reshape(len(lens), q_len, Hkv, Hq // Hkv, D)
    for b, L in enumerate(lens):
        k, v = R.seq_tokens(kd, bt[b], L, ps), R.seq_tokens(vd, bt[b], L, ps)
        for i in range(q_len):
            n = L - q_len + i + 1
            (p1, _, e1), (p2, _, e2) = (R.attend(qd[b, i], k, n, w, m * w) for m in range(2))
            ref = torch.einsum("hgn,nhd->hgd", p1 - p2, v[:n])
            tol = moved(p1, v[:n], e1) + moved(p2, v[:n], e2)
            if norm:
                inv = (ref.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
                # the norm's own change, first order; a fifth more for the second
                move = tol.square().mean(-1, keepdim=True).sqrt() * inv
                tol = (tol + ref.abs() * (move + 2.0 ** -20)) * inv * nw.double().abs() * 1.2
                ref = ref * inv * nw.double()
            ref, tol = ref.reshape(Hq, D), tol.reshape(Hq, D)
            bar = tol + R.rounding(ref.abs() + tol, od)
            off = (out[b, i] - ref).abs()
            assert (off <= bar).all(), (L, i, float((off / bar).max()))


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,ps,q_len", [(128, 8, 2, 16, 1), (64, 8, 2, 64, 1), (128, 16, 1, 32, 1), (128, 8, 2, 64, 4)])
def test_fp32_output_beside_the_totals_over_e4m3(fdlib, act, D, Hq, Hkv, ps, q_len):
    lens = [4, 5, 9, 40, 300]
    q, kp, vp, ks, vs, bt = setup("e4m3", act, lens, Hq, Hkv, D, ps, q_len, seed=D + Hq)
    dec = fd.PagedDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, out_dtype=torch.float32,
                                    track_weights=True)
    out, _, _ = dec.decode_weights(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                   torch.zeros(len(lens), Hkv, 300).cuda(), k_scale=ks.cuda(), v_scale=vs.cuda())
    torch.cuda.synchronize()
    dec.check()
    out = out.cpu().double().reshape(len(lens), q_len, Hkv, Hq // Hkv, D)
    kd, vd = R.values(kp, ks), R.values(vp, vs)
    qd = q.float().double().reshape(len(lens), q_len, Hkv, Hq // Hkv, D)
    for b, L in enumerate(lens):
        k, v = R.seq_tokens(kd, bt[b], L, ps), R.seq_tokens(vd, bt[b], L, ps)
        for i in range(q_len):
            n = L - q_len + i + 1
            p, _, err = R.attend(qd[b, i], k, n, D, 0)
            off, bar = (out[b, i] - torch.einsum("hgn,nhd->hgd", p, v[:n])).abs(), moved(p, v[:n], err)
            assert (off <= bar).all(), (L, i, float((off / bar).max()))

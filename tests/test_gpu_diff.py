"""Differential attention on the GPU against float64."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests import cache_ref as R
from tests.test_gpu_weights import setup

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def check(kv, act, lens, Hq, Hkv, D, ps, q_len=1, seed=0, norm="act", out_scale=0.2, out_dtype=None, lam=None, **opts):
    q, kp, vp, ks, vs, bt = setup(kv, act, lens, Hq, Hkv, D, ps, q_len, seed)
    gen = torch.Generator().manual_seed(seed + 7)
    lam = 0.2 + 0.6 * torch.rand(Hq, generator=gen) if lam is None else lam
    nw = None if norm is None else (1 + 0.3 * torch.randn(D, generator=gen)).to(torch.float32 if norm == "f32" else DT[act])
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    dec = fd.DiffDecoder.for_pools(g(q), g(kp), g(vp), g(bt), lens, out_dtype=out_dtype, **opts)
    out, lse = dec(g(q), g(kp), g(vp), g(bt), torch.tensor(lens, dtype=torch.int32).cuda(), g(lam), norm_weight=g(nw),
                   eps=1e-5, out_scale=out_scale, k_scale=g(ks), v_scale=g(vs))
    torch.cuda.synchronize()
    dec.check()
    B, G, w = len(lens), Hq // Hkv, D // 2
    od = DT[act] if out_dtype is None else out_dtype
    assert out.shape == q.shape and out.dtype == od and lse.shape == q.shape[:-1] + (2,)
    out, lse = out.cpu().double().reshape(B, q_len, Hq, D), lse.cpu().double().reshape(B, q_len, Hq, 2)
    kd, vd = R.values(kp, ks), R.values(vp, vs)
    qd = q.float().double().reshape(B, q_len, Hkv, G, D)
    lm = lam.double().reshape(Hkv, G, 1)
    for b, L in enumerate(lens):
        k, v = R.seq_tokens(kd, bt[b], L, ps), R.seq_tokens(vd, bt[b], L, ps)
        for i in range(q_len):
            n = max(0, L - q_len + i + 1)
            o, dev = torch.zeros(Hkv, G, D, dtype=torch.float64), torch.zeros(Hkv, G, D, dtype=torch.float64)
            for m in range(2):
                p, rl, err = R.attend(qd[b, i], k, n, w, m * w)
                got = lse[b, i, :, m].reshape(Hkv, G)
                if n == 0:
                    assert (got == -float("inf")).all()
                    continue
                assert ((got - rl).abs() <= err + 2.0 ** -20 + 2.0 ** -22 * rl.abs()).all()
                f = 1.0 if m == 0 else -lm
                o = o + f * torch.einsum("hgn,nhd->hgd", p, v[:n])
                # every term p v is off by p's rounding for the product (f16 2^-11, bf16 pairs
                # less), its exponent's error and the fp32 steps (2^-18)
                dev = dev + abs(f) * (2.0 ** -11 + 2 * err + 2.0 ** -18) * torch.einsum("hgn,nhd->hgd", p, v[:n].abs())
            if nw is not None:
                inv = (o.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
                scale = nw.double() * out_scale
                # the norm's own change: at most rms(dev) * inv of the value, first order
                move = dev.square().mean(-1, keepdim=True).sqrt() * inv
                ref, tol = o * inv * scale, (dev + o.abs() * (move + 2.0 ** -20)) * inv * scale.abs() * 1.2
            else:
                ref, tol = o * out_scale, dev * abs(out_scale)
            ref, tol = ref.reshape(Hq, D), tol.reshape(Hq, D)
            bar = tol + R.rounding(ref.abs() + tol, od)
            assert ((out[b, i] - ref).abs() <= bar).all(), float(((out[b, i] - ref).abs() - bar).max())


@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 16, 8), (128, 10, 2), (64, 24, 2), (128, 16, 1)])
def test_types_and_groups(fdlib, kv, act, D, Hq, Hkv):
    check(kv, act, [1, 16, 300, 0, 77], Hq, Hkv, D, 16, seed=D + Hq)


@pytest.mark.parametrize("norm,out_scale,out_dtype", [(None, 1.0, None), ("f32", 0.5, torch.float32), ("act", -2.0, None),
                                                      (None, 0.0, torch.float32)])
def test_norm_and_output_types(fdlib, norm, out_scale, out_dtype):
    check("bf16", "bf16", [50, 700], 8, 2, 128, 32, norm=norm, out_scale=out_scale, out_dtype=out_dtype)
    check("f16", "f16", [50, 700], 8, 2, 64, 32, norm=norm, out_scale=out_scale, out_dtype=out_dtype)


@pytest.mark.parametrize("opts", [dict(num_splits=1), dict(num_splits=3), dict(num_splits=12),
                                  dict(num_splits=3, fuse_merge=0), dict(tile_tokens=64, ctas_per_sm=2),
                                  dict(tile_tokens=128, ctas_per_sm=2)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_plan_shapes(fdlib, kv, opts):
    if kv == "bf16" and opts.get("tile_tokens") == 128:
        opts = dict(tile_tokens=128)  # two CTAs of 128-token stages fit an SM with E4M3 only
    check(kv, "bf16", [900, 64, 2049, 1], 16, 4, 128, 64, seed=2, **opts)
    check(kv, "bf16", [900, 64, 513, 0], 3, 3, 64, 16, seed=3, out_dtype=torch.float32, **opts)


@pytest.mark.parametrize("kv,q_len,Hq,Hkv", [("bf16", 4, 8, 2), ("f16", 3, 5, 1), ("e4m3", 5, 8, 2), ("bf16", 2, 3, 3)])
def test_query_tokens(fdlib, kv, q_len, Hq, Hkv):
    check(kv, "f16" if kv == "f16" else "bf16", [q_len, 40, 700], Hq, Hkv, 128, 16, q_len=q_len, seed=q_len)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,ps,q_len", [(128, 8, 2, 64, 4), (64, 4, 1, 32, 6), (128, 2, 1, 128, 3), (128, 3, 3, 64, 2)])
def test_query_tokens_over_e4m3_pages_of_256_token_stages(fdlib, act, D, Hq, Hkv, ps, q_len):
    """Causal limits that fall in either sub-tile of a warp, lengths around a stage."""
    check("e4m3", act, [q_len, 255, 256, 257, 520, 1000], Hq, Hkv, D, ps, q_len=q_len, seed=q_len)
    check("e4m3", act, [2000, q_len + 1], Hq, Hkv, D, ps, q_len=q_len, seed=q_len, num_splits=3, out_dtype=torch.float32)


def test_long_split_sequence(fdlib):
    check("bf16", "bf16", [20011], 8, 2, 128, 64, seed=4)
    check("e4m3", "bf16", [9000, 16], 8, 2, 128, 128, seed=5)


def test_equal_maps_cancel(fdlib):
    """q1 = q2 over k1 = k2 with lambda = 1: nothing is left."""
    lens = [1, 200]
    q, kp, vp, _, _, bt = setup("bf16", "bf16", lens, 4, 2, 128, 16)
    q[..., 64:], kp[..., 64:] = q[..., :64], kp[..., :64]
    dec = fd.DiffDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, out_dtype=torch.float32)
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = dec(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), dl, torch.ones(4).cuda())
    torch.cuda.synchronize()
    # both maps go through the same sums: a few fp32 steps of |V| <= 6
    assert float(out.abs().max()) <= 6 * 2.0 ** -18
    assert float((lse[..., 0] - lse[..., 1]).abs().max()) <= 2.0 ** -18
    zero, _ = dec(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), dl, torch.zeros(4).cuda(), want_lse=False)
    assert float(zero.abs().max()) > 0.1


def test_graph_replay_and_other_stream(fdlib):
    lens = [700, 33]
    q, kp, vp, _, _, bt = (None if t is None else t.cuda() for t in setup("bf16", "bf16", lens, 16, 4, 128, 16))
    dl, lam = torch.tensor(lens, dtype=torch.int32).cuda(), torch.rand(16).cuda()
    dec = fd.DiffDecoder.for_pools(q, kp, vp, bt, lens)
    out, lse = dec(q, kp, vp, bt, dl, lam)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out2, lse2 = dec(q, kp, vp, bt, dl, lam)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out3, _ = dec(q, kp, vp, bt, dl, lam, stream=side)
    side.synchronize()
    assert torch.equal(out, out3)
    dec.check()


def test_length_past_the_plan_is_flagged(fdlib):
    lens = [100]
    q, kp, vp, _, _, bt = (None if t is None else t.cuda() for t in setup("bf16", "bf16", [4000], 4, 2, 128, 16))
    dec = fd.DiffDecoder.for_pools(q, kp, vp, bt, lens)
    dec(q, kp, vp, bt, torch.tensor([3999], dtype=torch.int32).cuda(), torch.rand(4).cuda())
    with pytest.raises(_lib.FdError) as e:
        dec.check()
    assert e.value.code == _lib.FD_ERR_CAPACITY


@pytest.mark.parametrize("mode", ["diff", "weights"])
@pytest.mark.parametrize("opts", [dict(), dict(num_splits=3), dict(tile_tokens=128, ctas_per_sm=2), dict(tile_tokens=64)])
def test_e4m3_pages_of_very_different_scales(fdlib, mode, opts):
    """V scales from 2^-10 to 2^10, some zero."""
    lens, D, ps = [1000, 37, 300], 128, 32
    q, kp, vp, ks, vs, bt = setup("e4m3", "bf16", lens, 8, 2, D, ps, seed=9)
    gen = torch.Generator().manual_seed(3)
    vs = torch.exp2(torch.rand(vs.shape, generator=gen) * 20 - 10) / 448 * (torch.rand(vs.shape, generator=gen) > 0.1)
    g = lambda t: t.cuda()  # noqa: E731
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    if mode == "diff":
        dec = fd.DiffDecoder.for_pools(g(q), g(kp), g(vp), g(bt), lens, out_dtype=torch.float32, **opts)
        out, _ = dec(g(q), g(kp), g(vp), g(bt), dl, torch.full((8,), 0.5).cuda(), k_scale=g(ks), v_scale=g(vs))
    else:
        dec = fd.PagedDecoder.for_pools(g(q), g(kp), g(vp), g(bt), lens, out_dtype=torch.float32, track_weights=True, **opts)
        out, _, _ = dec.decode_weights(g(q), g(kp), g(vp), g(bt), dl, torch.zeros(3, 2, 1000).cuda(), k_scale=g(ks),
                                       v_scale=g(vs))
    torch.cuda.synchronize()
    dec.check()
    out = out.cpu().double().reshape(3, 2, 4, D)
    kd, vd = R.values(kp, ks), R.values(vp, vs)
    for b, L in enumerate(lens):
        k, v = R.seq_tokens(kd, bt[b], L, ps), R.seq_tokens(vd, bt[b], L, ps)
        qd = q[b].float().double().reshape(2, 4, D)
        ref, tol = torch.zeros(2, 4, D, dtype=torch.float64), torch.zeros(2, 4, D, dtype=torch.float64)
        for m, f in (((0, 1.0), (1, -0.5)) if mode == "diff" else ((0, 1.0),)):
            width = D // 2 if mode == "diff" else D
            p, _, err = R.attend(qd, k, L, width, m * width)
            ref += f * torch.einsum("hgn,nhd->hgd", p, v)
            # a weight's rounding for the product (2^-11) and its exponent's error, the fp32
            # steps (2^-18), and f16's floor of 2^-25
            tol += abs(f) * ((2.0 ** -11 + 2 * err + 2.0 ** -18) * torch.einsum("hgn,nhd->hgd", p, v.abs()) +
                             2.0 ** -25 * v.abs().sum(0)[:, None])
        assert ((out[b] - ref).abs() <= tol).all(), float(((out[b] - ref).abs() / tol).max())

"""append_kv_norm on the GPU against float64: norms, rotations, paged writes,
strides, padded batches, separate positions, device error flags."""
import numpy as np
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests import cache_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def tables(max_pos, half, base=10000.0):
    ang = np.arange(max_pos)[:, None] / base ** (np.arange(half) / max(half, 1))
    return torch.from_numpy(np.cos(ang).astype(np.float32)), torch.from_numpy(np.sin(ang).astype(np.float32))


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16)


def check(kv, act, B, T, Hq, Hkv, D, ps, rd, interleaved=False, wt="act", fused=True, ragged=None, lens=None,
          positions=None, use_q=True, in_place=False, seed=0, mult=1.0):
    gen = torch.Generator().manual_seed(seed)
    cache, act = DT[kv], DT[act]
    lens = [int(x) for x in torch.randint(0, 3 * ps, (B,), generator=gen)] if lens is None else lens
    new = [T] * B if ragged is None else ragged
    bt, pages, _ = R.make_table(gen, [a + n for a, n in zip(lens, new)], ps)
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, cache)
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, cache)
    lead = (B, T) if T > 1 or ragged is not None else (B,)
    if fused:
        rows = (torch.randn(lead + ((Hq + 2 * Hkv) * D + 8,), generator=gen) * mult).to(act).cuda()
        cut = [Hq * D, Hkv * D, Hkv * D, 8]
        q, k, v, _ = rows.split(cut, -1)
        q, k, v = q.unflatten(-1, (Hq, D)), k.unflatten(-1, (Hkv, D)), v.unflatten(-1, (Hkv, D))
    else:
        q, k, v = ((torch.randn(lead + (h, D), generator=gen) * mult).to(act).cuda() for h in (Hq, Hkv, Hkv))
    w = None if wt is None else [(1 + 0.3 * torch.randn(D, generator=gen)).to(torch.float32 if wt == "f32" else act)
                                 for _ in range(2)]
    max_pos = max(l + n for l, n in zip(lens, new)) + 100
    cos, sin = tables(max_pos, rd // 2) if rd else (None, None)
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    gk, gv = kp.cuda(), vp.cuda()
    src = [t.detach().cpu().double() for t in (q, k, v)]
    marker = torch.full(lead + (Hq, D), 7.0, dtype=act, device="cuda")
    q_out = q if in_place else marker
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fd.append_kv_norm(q if use_q else None, k, v, gk, gv, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            q_weight=g(w[0]) if w else None, k_weight=g(w[1]) if w else None, eps=1e-5, rotary_cos=g(cos),
                            rotary_sin=g(sin), interleaved=interleaved,
                            positions=None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda(),
                            new_lens=None if ragged is None else torch.tensor(ragged, dtype=torch.int32).cuda(),
                            k_scale=g(ks), v_scale=g(vs), q_out=q_out if use_q else None, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    sq, sk, sv = (t.reshape((B, T) + t.shape[-2:]) for t in src)
    live = torch.zeros(pages, ps, dtype=torch.bool)
    hk, hv = gk.cpu(), gv.cpu()
    out = got.cpu().reshape(B, T, Hq, D) if use_q else None
    for b in range(B):
        n, at = new[b], lens[b]
        p0 = at if positions is None else positions[b]
        c, s = (cos[p0:p0 + n], sin[p0:p0 + n]) if rd else (None, None)
        pg = bt[b, torch.arange(at, at + n) // ps].long()
        sl = torch.arange(at, at + n) % ps
        live[pg, sl] = True
        rk, ek = R.norm_rotate(sk[b, :n], w[1] if w else None, 1e-5, c, s, interleaved)
        rv, ev = sv[b, :n], torch.zeros_like(sv[b, :n])
        for ref, err, pool, scale in ((rk, ek, hk, ks), (rv, ev, hv, vs)):
            x = pool.float()[pg, sl].double()
            if scale is not None:  # in code units; the division adds 2^-24
                sc = scale[pg].double()[..., None]
                ref, err = (ref / sc).clamp(-448, 448), err / sc + 2.0 ** -23 * (ref / sc).abs()
            assert ((x - ref).abs() <= err * 1.1 + R.rounding(ref.abs() + err, cache)).all()
        if use_q:
            rq, eq = R.norm_rotate(sq[b, :n], w[0] if w else None, 1e-5, c, s, interleaved)
            x = out[b, :n].double()
            assert ((x - rq).abs() <= eq + R.rounding(rq.abs() + eq, act)).all()
            if not in_place:
                assert (out[b, n:] == 7.0).all()
            else:
                assert torch.equal(out[b, n:].double(), sq[b, n:])
    # nothing else of the pools changed
    assert torch.equal(bits(hk)[~live], bits(kp)[~live]) and torch.equal(bits(hv)[~live], bits(vp)[~live])


@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot", ["none", "full", "pairs", "half", "odd", "odd_pairs"])
def test_types_and_rotations(fdlib, kv, act, D, rot):
    rd = {"none": 0, "full": D, "pairs": D, "half": D // 2, "odd": D // 4 + 2, "odd_pairs": D // 4 + 2}[rot]
    check(kv, act, B=3, T=1, Hq=6, Hkv=3, D=D, ps=16, rd=rd, interleaved=rot.endswith("pairs"), seed=len(rot) + D)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rd", [(64, 2), (64, 8), (64, 24), (64, 62), (128, 40), (128, 120), (128, 126), (128, 4)])
def test_partial_rotations(fdlib, D, rd, interleaved):
    check("bf16", "bf16", B=2, T=5, Hq=4, Hkv=2, D=D, ps=16, rd=rd, interleaved=interleaved, seed=rd)
    check("e4m3", "f16", B=2, T=1, Hq=2, Hkv=1, D=D, ps=16, rd=rd, interleaved=interleaved, seed=rd + 1)


def test_tables_and_weights_off_alignment(fdlib):
    """Cosines, sines and norm weights that start 4 (2) bytes off 16: read element by element."""
    gen = torch.Generator().manual_seed(7)
    B, H, D, ps = 2, 3, 128, 16
    bt, pages, _ = R.make_table(gen, [30] * B, ps)
    kp = torch.zeros(pages, ps, H, D, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(B, H, D, generator=gen).bfloat16().cuda()
    cos, sin = (t.cuda() for t in tables(64, D // 2))
    w = (1 + torch.randn(D, generator=gen)).bfloat16().cuda()
    lens = torch.tensor([20, 3], dtype=torch.int32).cuda()
    off = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
    for interleaved in (False, True):
        ref = fd.append_kv_norm(x, x, x, kp, kp.clone(), bt.cuda(), lens, q_weight=w, k_weight=w, rotary_cos=cos,
                                rotary_sin=sin, interleaved=interleaved)
        one = kp.clone()
        got = fd.append_kv_norm(x, x, x, kp, kp.clone(), bt.cuda(), lens, q_weight=off(w), k_weight=off(w),
                                rotary_cos=off(cos), rotary_sin=off(sin), interleaved=interleaved)
        torch.cuda.synchronize()
        assert off(cos).data_ptr() % 16 == 4 and off(w).data_ptr() % 4 == 2
        assert torch.equal(bits(ref), bits(got)) and torch.equal(bits(one), bits(kp))


@pytest.mark.parametrize("B,T,Hq,Hkv,ps", [(1, 1, 1, 1, 16), (1, 1, 32, 8, 64), (2, 5, 7, 7, 48), (1, 300, 5, 1, 16),
                                           (40, 33, 12, 2, 32), (700, 1, 3, 1, 16)])
def test_sizes(fdlib, B, T, Hq, Hkv, ps):
    check("bf16", "bf16", B, T, Hq, Hkv, 128, ps, rd=128, seed=B)
    check("e4m3", "bf16", B, T, Hq, Hkv, 64, ps, rd=34, seed=B + 1)


@pytest.mark.parametrize("rot", ["none", "full", "pairs", "half", "odd"])
@pytest.mark.parametrize("kv,D", [("bf16", 128), ("e4m3", 64)])
def test_many_tokens(fdlib, kv, D, rot):
    """Enough tokens that a warp takes several steps of a token, or all of them."""
    rd = {"none": 0, "full": D, "pairs": D, "half": D // 2, "odd": D // 4 + 2}[rot]
    il = rot == "pairs"
    check(kv, "bf16", 3, 700, 32, 8, D, 16, rd=rd, interleaved=il, ragged=[700, 0, 333], lens=[0, 5, 16])
    check(kv, "bf16", 2, 2500, 9, 3, D, 64, rd=rd, interleaved=il, lens=[7, 0], seed=1)
    check(kv, "bf16", 6, 2100, 5, 1, D, 32, rd=rd, interleaved=il, ragged=[2100, 1, 2099, 0, 1000, 5], lens=[0] * 6, seed=2)


def test_padded_batch_with_empty_rows(fdlib):
    check("bf16", "bf16", 5, 37, 8, 2, 128, 16, rd=128, ragged=[0, 37, 1, 16, 0])
    check("f16", "f16", 3, 1, 4, 4, 64, 16, rd=64, ragged=[1, 0, 1])


def test_separate_tensors_fp32_weights_and_positions(fdlib):
    check("bf16", "bf16", 4, 9, 8, 2, 128, 16, rd=64, wt="f32", fused=False, positions=[0, 90, 3, 40])
    check("f16", "f16", 4, 1, 8, 2, 128, 16, rd=0, wt="f32", fused=False)


def test_in_place_and_without_queries(fdlib):
    check("bf16", "bf16", 4, 9, 8, 2, 128, 16, rd=128, in_place=True, ragged=[9, 0, 4, 9])
    check("bf16", "bf16", 4, 9, 8, 2, 128, 16, rd=128, fused=False, in_place=True)
    check("e4m3", "bf16", 4, 9, 8, 2, 128, 16, rd=128, use_q=False)


def test_large_and_small_values(fdlib):
    """E4M3 codes saturate; tiny rows are normed up."""
    check("e4m3", "bf16", 2, 3, 4, 2, 128, 16, rd=128, wt=None, mult=100.0)
    check("bf16", "bf16", 2, 3, 4, 2, 128, 16, rd=128, mult=2.0 ** -20)
    check("f16", "f16", 2, 3, 4, 2, 64, 16, rd=64, mult=2.0 ** -10)


@pytest.mark.parametrize("kv,interleaved,rd", [("bf16", 0, 128), ("bf16", 1, 64), ("e4m3", 0, 128), ("f16", 0, 34)])
def test_without_norm_equals_the_rotary_append(fdlib, kv, interleaved, rd):
    """No norm weights, one token: bit for bit fd_append_kv_rotary."""
    gen = torch.Generator().manual_seed(3)
    B, Hq, Hkv, D, ps = 3, 8, 2, 128, 16
    act = DT["f16"] if kv == "f16" else DT["bf16"]
    lens = [0, 17, 40]
    bt, pages, _ = R.make_table(gen, [n + 1 for n in lens], ps)
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    q, k, v = (torch.randn(B, h, D, generator=gen).to(act).cuda() for h in (Hq, Hkv, Hkv))
    cos, sin = (t.cuda() for t in tables(64, rd // 2))
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    a, b = [kp.cuda(), vp.cuda()], [kp.cuda(), vp.cuda()]
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    q1 = fd.append_kv_norm(q, k, v, *a, bt.cuda(), dl, rotary_cos=cos, rotary_sin=sin, interleaved=bool(interleaved),
                           k_scale=g(ks), v_scale=g(vs))
    prob = _lib.make_problem(B, Hq, Hkv, D, ps, bt.shape[1], pages, act, DT[kv])
    q2 = q.clone()
    _lib.fd_append_kv_rotary(prob, k, v, *b, g(ks), g(vs), bt.cuda(), dl, cos, sin, interleaved=bool(interleaved),
                             q_inout=q2)
    torch.cuda.synchronize()
    assert torch.equal(bits(q1), bits(q2))
    assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))


def test_device_errors_are_flagged_and_skipped(fdlib):
    D, ps = 64, 16
    kp = torch.zeros((4, ps, 2, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    x = torch.ones((2, 3, 2, D), dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bt = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    status = i32(0)
    kw = dict(q_weight=None, k_weight=None, status=status)
    # row 0 runs past its table after one token, row 1 into an unused entry after two
    q = fd.append_kv_norm(x, x, x, kp, vp, bt, i32(31, 14), **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.FD_DEV_BAD_PAGE
    assert torch.equal(q, x)
    want = torch.zeros(4, ps, dtype=torch.bool, device="cuda")
    want[1, 15] = want[2, 14] = want[2, 15] = True
    assert torch.equal(kp.float().sum((2, 3)) > 0, want) and torch.equal(vp.float().sum((2, 3)) > 0, want)
    # a negative length
    status.zero_()
    kp.zero_()
    fd.append_kv_norm(x, x, x, kp, vp, bt, i32(-2, 0), **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.FD_DEV_BAD_PAGE
    assert int((kp.float().sum((2, 3)) > 0).sum()) == 3
    # positions outside the table of angles: those tokens are skipped
    status.zero_()
    kp.zero_()
    cos = torch.ones(4, D // 2, device="cuda")
    q = torch.zeros_like(x)
    fd.append_kv_norm(x, x, x, kp, vp, bt, i32(0, 0), rotary_cos=cos, rotary_sin=cos * 0, positions=i32(2, -1), q_out=q,
                      **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.FD_DEV_CAPACITY
    assert (q.float().sum((2, 3)) > 0).tolist() == [[True, True, False], [False, True, True]]
    assert int((kp.float().sum((2, 3)) > 0).sum()) == 4
    # token counts outside [0, T]
    status.zero_()
    kp.zero_()
    fd.append_kv_norm(x, x, x, kp, vp, bt, i32(0, 0), new_lens=i32(4, -1), **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.FD_DEV_CAPACITY and not kp.float().abs().sum().item()


def test_graph_replay_and_other_stream(fdlib):
    gen = torch.Generator().manual_seed(5)
    B, Hq, Hkv, D, ps = 4, 8, 2, 128, 16
    bt, pages, _ = R.make_table(gen, [40] * B, ps)
    bt = bt.cuda()
    kp, vp = (torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.randn(B, h, D, generator=gen).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    lens = torch.full((B,), 20, dtype=torch.int32, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    call = lambda **kw: fd.append_kv_norm(q, k, v, kp, vp, bt, lens, q_weight=w, k_weight=w, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ref = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q_out=out)
    for i in range(3):
        graph.replay()
        lens += 1
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    for b in range(B):
        rows = kp[bt[b, torch.arange(20, 23, device="cuda") // ps].long(), torch.arange(20, 23, device="cuda") % ps]
        assert torch.equal(rows[0], rows[1]) and torch.equal(rows[0], rows[2]) and rows.float().abs().sum() > 0

"""decode_weights on the GPU: the totals of attention weights against float64,
the output and lse against the plain decode's parity bar."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests import cache_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
TOL_OUT = {"f16": 2e-3, "bf16": 2e-3, "e4m3": 3e-2}


def setup(kv, act, lens, Hq, Hkv, D, ps, q_len=1, seed=0, cols=0):
    gen = torch.Generator().manual_seed(seed)
    bt, pages, _ = R.make_table(gen, lens, ps, pad_cols=cols)
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    lead = (len(lens),) if q_len == 1 else (len(lens), q_len)
    q = torch.randn(lead + (Hq, D), generator=gen).to(DT[act])
    return q, kp, vp, ks, vs, bt


def reference(q, kp, vp, ks, vs, bt, lens, ps, q_len):
    """Per sequence: out, lse [q_len, Hq(, D)], weights [Hkv, L], score error."""
    B, Hkv, D = len(lens), kp.shape[2], kp.shape[3]
    kd, vd = R.values(kp, ks), R.values(vp, vs)
    qd = q.float().double().reshape(B, q_len, Hkv, -1, D)
    res = []
    for b, L in enumerate(lens):
        k, v = R.seq_tokens(kd, bt[b], L, ps), R.seq_tokens(vd, bt[b], L, ps)
        w, outs, lses, err = torch.zeros(Hkv, L, dtype=torch.float64), [], [], 0.0
        for i in range(q_len):
            n = max(0, L - q_len + i + 1)
            p, lse, e = R.attend(qd[b, i], k, n, D, 0)
            w[:, :n] += p.sum(1)
            outs.append(torch.einsum("hgn,nhd->hgd", p, v[:n]).flatten(0, 1))
            lses.append(lse.flatten())
            err = max(err, e)
        res.append((torch.stack(outs), torch.stack(lses), w, err))
    return res


def check(kv, act, lens, Hq, Hkv, D, ps, q_len=1, seed=0, mode="separate", room=None, out_dtype=None, **opts):
    q, kp, vp, ks, vs, bt = setup(kv, act, lens, Hq, Hkv, D, ps, q_len, seed)
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    N = max(lens) + 5 if room is None else room
    w0 = torch.rand(len(lens), Hkv, N, generator=torch.Generator().manual_seed(seed + 1)) * 3
    dec = fd.PagedDecoder.for_pools(g(q), g(kp), g(vp), g(bt), lens, track_weights=True, out_dtype=out_dtype, **opts)
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    args = (g(q), g(kp), g(vp), g(bt), dl)
    win = None if mode == "fresh" else g(w0)
    wout = {"separate": lambda: torch.full_like(win, 9.0), "in place": lambda: None,
            "fresh": lambda: torch.full(w0.shape, 9.0, device="cuda")}[mode]()
    out, lse, total = dec.decode_weights(*args, win, weights_out=wout, k_scale=g(ks), v_scale=g(vs))
    torch.cuda.synchronize()
    dec.check()
    if mode == "in place":
        assert total is win
    if mode == "separate":
        assert torch.equal(win.cpu(), w0)
    total, out, lse = total.cpu().double(), out.cpu().double(), lse.cpu().double()
    B = len(lens)
    out, lse = out.reshape(B, q_len, Hq, D), lse.reshape(B, q_len, Hq)
    G = Hq // Hkv
    for b, (ro, rl, rw, err) in enumerate(reference(q, kp, vp, ks, vs, bt, lens, ps, q_len)):
        L = lens[b]
        # lse: an average of score errors, the fp32 sum (2^-20 covers its steps) and its logarithm
        tol_l = err + 2.0 ** -20 + 2.0 ** -22 * rl.abs()
        inf = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse[b]), inf)
        assert ((lse[b] - rl).abs()[~inf] <= tol_l[~inf]).all()
        od = DT[act] if out_dtype is None else out_dtype
        assert ((out[b] - ro).abs() <= TOL_OUT[kv] + R.rounding(ro, od)).all()
        # a weight is off by exp's error (2^-21) and its exponent's: score, lse and
        # their difference in log2 units (2^-23 of each); then R rounded additions
        rel = 2 * err + 2.0 ** -19 + 2.0 ** -21 * float(rl[~inf].abs().max() if (~inf).any() else 0) + G * q_len * 2.0 ** -24
        base = torch.zeros(Hkv, L, dtype=torch.float64) if mode == "fresh" else w0[b, :, :L].double()
        ref = base + rw
        assert ((total[b, :, :L] - ref).abs() <= rw * rel + 1e-30 + 2.0 ** -24 * ref).all()
        tail = w0[b, :, L:].double() if mode == "in place" else torch.full_like(total[b, :, L:], 9.0)
        assert torch.equal(total[b, :, L:], tail)


@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 32, 8), (128, 10, 2), (64, 24, 2)])
def test_types_and_groups(fdlib, kv, act, D, Hq, Hkv):
    check(kv, act, [1, 16, 300, 77], Hq, Hkv, D, 16, seed=D + Hq)


@pytest.mark.parametrize("mode", ["separate", "in place", "fresh"])
def test_in_place_and_fresh(fdlib, mode):
    check("bf16", "bf16", [0, 5, 129, 1000, 0], 8, 2, 128, 32, mode=mode)


@pytest.mark.parametrize("opts", [dict(num_splits=1), dict(num_splits=3), dict(num_splits=7),
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


def test_long_split_sequence(fdlib):
    check("bf16", "bf16", [20011], 8, 2, 128, 64, seed=4)
    check("e4m3", "bf16", [9000, 16], 16, 2, 128, 128, seed=5)


def test_weights_of_a_step_sum_to_the_query_heads(fdlib):
    """Without earlier totals a KV head's weights sum to its number of query rows."""
    lens = [7, 500]
    q, kp, vp, ks, vs, bt = setup("bf16", "bf16", lens, 12, 4, 64, 16)
    dec = fd.PagedDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, track_weights=True)
    w = torch.zeros(2, 4, 512, device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    for step in range(1, 4):
        dec.decode_weights(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), dl, w)
        torch.cuda.synchronize()
        # 500 weights of relative error 2^-15 at most (see above), three times
        assert torch.allclose(w.double().sum(-1).cpu(), torch.full((2, 4), 3.0 * step, dtype=torch.float64), rtol=2e-4)


def test_short_rows_of_totals_are_flagged(fdlib):
    lens = [50, 20]
    q, kp, vp, ks, vs, bt = setup("bf16", "bf16", lens, 8, 2, 64, 16)
    dec = fd.PagedDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, track_weights=True)
    w = torch.full((3, 2, 32), 5.0, device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    dec.decode_weights(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), dl, w[:2])
    with pytest.raises(_lib.FdError) as e:
        dec.check()
    assert e.value.code == _lib.FD_ERR_CAPACITY
    assert (w[2] == 5.0).all() and (w[1, :, 20:] == 5.0).all() and (w[1, :, :20] > 5.0).all()


def test_graph_replay_and_other_stream(fdlib):
    lens = [700, 33]
    q, kp, vp, ks, vs, bt = (None if t is None else t.cuda() for t in setup("bf16", "bf16", lens, 16, 4, 128, 16))
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    dec = fd.PagedDecoder.for_pools(q, kp, vp, bt, lens, track_weights=True)
    w = torch.zeros(2, 4, 700, device="cuda")
    out, lse, one = dec.decode_weights(q, kp, vp, bt, dl, None, weights_out=torch.zeros_like(w))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out2, lse2, _ = dec.decode_weights(q, kp, vp, bt, dl, w)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    acc = torch.zeros_like(w)
    for _ in range(3):
        acc += one
    assert torch.equal(w, acc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out3, _, w3 = dec.decode_weights(q, kp, vp, bt, dl, None, weights_out=torch.zeros_like(w), stream=side)
    side.synchronize()
    assert torch.equal(out, out3) and torch.equal(one, w3)
    dec.check()

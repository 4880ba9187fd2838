"""evict_kv on the GPU: what stays, where it goes, and what is left alone."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests import cache_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16)


def check(kv, lens, Hkv, D, ps, budget, sinks, recent, fresh, seed=0, w=None, weights="out", equal_scales=False):
    gen = torch.Generator().manual_seed(seed)
    n_new = [min(L, budget) for L in lens]
    bt, pages, spare = R.make_table(gen, lens, ps, extra=sum(-(-n // ps) for n in n_new) + 1, pad_cols=1)
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    if equal_scales and ks is not None:
        ks, vs = torch.full_like(ks, 0.25), torch.full_like(vs, 0.25)
    dst = None
    if fresh:
        dst, at = torch.full_like(bt, -1), 0
        for b, n in enumerate(n_new):
            m = -(-n // ps)
            dst[b, :m] = spare[at:at + m]
            at += m
    B, N = len(lens), max(max(lens), 1) + 3
    if w is None:
        w = torch.rand(B, Hkv, N, generator=gen) ** 4 * (torch.rand(B, Hkv, N, generator=gen) > 0.1)
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    gk, gv, gw = kp.cuda(), vp.cuda(), w.cuda()
    wout = {"out": lambda: torch.full_like(gw, 9.0), "in place": lambda: gw, "none": lambda: None}[weights]()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n, kept = fd.evict_kv(gk, gv, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), gw, budget, sinks, recent,
                          dst_table=g(dst), weights_out=wout, k_scale=g(ks), v_scale=g(vs), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert n.tolist() == n_new
    kept, hk, hv = kept.cpu(), gk.cpu(), gv.cpu()
    written = torch.zeros(pages, ps, dtype=torch.bool)
    to_table = bt if dst is None else dst
    for b, L in enumerate(lens):
        for h in range(Hkv):
            keep = R.evict(w[b, h], L, budget, sinks, recent)
            m = len(keep)
            assert kept[b, h, :m].tolist() == keep.tolist()
            assert (kept[b, h, m:] == -1).all()
            j = torch.arange(m)
            p0, s0 = bt[b, keep // ps].long(), keep % ps
            p1, s1 = to_table[b, j // ps].long(), j % ps
            written[p1, s1] = True
            for old, new, sc in ((kp, hk, ks), (vp, hv, vs)):
                if sc is None:
                    assert torch.equal(bits(new)[p1, s1, h], bits(old)[p0, s0, h])
                    continue
                a, z = sc[p0, h][:, None], sc[p1, h][:, None]
                x = old.view(torch.uint8)[p0, s0, h].view(DT[kv]).float()
                want = (x * (a / z)).clamp(-448, 448).to(DT[kv]).view(torch.uint8)
                same = (a / z == 1).expand_as(x)
                want = torch.where(same, old.view(torch.uint8)[p0, s0, h], want)
                assert torch.equal(new.view(torch.uint8)[p1, s1, h], want)
            if wout is not None:
                row = wout[b, h].cpu()
                assert torch.equal(row[:m].nan_to_num(77.0), w[b, h, keep].nan_to_num(77.0))
                assert (row[m:L] == 0).all()
                rest = w[b, h, L:] if weights == "in place" else torch.full_like(row[L:], 9.0)
                assert torch.equal(row[L:].nan_to_num(77.0), rest.nan_to_num(77.0))
    if weights != "in place":
        assert torch.equal(gw.cpu().nan_to_num(77.0), w.nan_to_num(77.0))
    assert torch.equal(bits(hk)[~written], bits(kp)[~written]) and torch.equal(bits(hv)[~written], bits(vp)[~written])


@pytest.mark.parametrize("fresh", [False, True], ids=["in place", "fresh pages"])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_types(fdlib, fresh, kv, D):
    check(kv, [0, 1, 40, 41, 100, 333], 3, D, 16, budget=40, sinks=4, recent=10, fresh=fresh, seed=D)


@pytest.mark.parametrize("fresh", [False, True], ids=["in place", "fresh pages"])
@pytest.mark.parametrize("ps,budget,sinks,recent", [(16, 1, 0, 0), (16, 1, 1, 0), (48, 1, 0, 1), (32, 60, 60, 0),
                                                    (64, 60, 0, 60), (16, 64, 30, 34), (128, 500, 0, 0),
                                                    (16, 499, 0, 1), (32, 1000, 7, 600)])
def test_budgets(fdlib, fresh, ps, budget, sinks, recent):
    check("bf16", [500, 1100, 61, 1001], 2, 64, ps, budget, sinks, recent, fresh, seed=budget)


@pytest.mark.parametrize("fresh", [False, True], ids=["in place", "fresh pages"])
def test_long_rows(fdlib, fresh):
    """Several tiles of the scan, a steady state one token over its budget among them."""
    check("bf16", [9001, 8192, 12289], 2, 64, 64, 8191, 4, 1000, fresh, seed=1)
    check("e4m3", [20000], 1, 128, 128, 9999, 16, 0, fresh, seed=2)


@pytest.mark.parametrize("fresh,weights", [(False, "in place"), (True, "out")])
def test_rows_of_several_rounds(fdlib, fresh, weights):
    """More tokens than the selecting CTAs hold at once: one row longer than a
    cluster's tiles, and so many rows that each has one CTA."""
    check("f16", [140001], 1, 64, 64, 90000, 4, 1000, fresh, seed=1, weights=weights)
    check("bf16", [140001], 1, 64, 128, 60000, 0, 0, fresh, seed=2, weights=weights, w=torch.full((1, 1, 140004), 0.25))
    check("e4m3", [9000 + i for i in range(39)], 4, 64, 64, 7000, 4, 100, fresh, seed=3, weights=weights)


@pytest.mark.parametrize("weights", ["out", "in place", "none"])
def test_weights_out(fdlib, weights):
    check("bf16", [700, 5, 90], 2, 64, 16, 77, 3, 20, False, weights=weights)


def test_many_heads_in_place(fdlib):
    """Enough sequences that a CTA moves whole rows of K or V."""
    check("bf16", [130] * 60, 3, 128, 16, 100, 1, 7, False, seed=3)
    check("e4m3", [130] * 60, 3, 64, 16, 100, 1, 7, False, seed=4)


def test_equal_scales_keep_the_codes(fdlib):
    check("e4m3", [300, 64], 2, 128, 32, 50, 2, 9, False, equal_scales=True)


def test_ties_and_unusual_weights(fdlib):
    """All equal: the lowest indices stay.  Infinities, NaN, signed zeros, negatives."""
    check("bf16", [200], 2, 64, 16, 90, 5, 11, False, w=torch.full((1, 2, 203), 0.5))
    check("bf16", [200], 1, 64, 16, 90, 0, 0, True, w=torch.zeros(1, 1, 203))
    inf, nan = float("inf"), float("nan")
    base = torch.tensor([inf, -inf, nan, 0.0, -0.0, 1e-45, -1.0, 3.0, nan, 2.0, -0.0, 0.0, inf, -nan, 1.0, 3.4e38])
    w = base.repeat(13)[:203].view(1, 1, -1).clone()
    for budget in (10, 26, 27, 60, 65, 100, 130, 170, 199):
        check("bf16", [200], 1, 64, 16, budget, 0, 0, False, w=w)


def test_device_errors_leave_the_sequence(fdlib):
    gen = torch.Generator().manual_seed(0)
    kp, _ = R.make_pool(gen, 12, 16, 2, 64, torch.bfloat16)
    gk, gv = kp.cuda(), kp.cuda().clone()
    bt = torch.arange(12, dtype=torch.int32).view(3, 4).cuda()
    w = torch.rand(3, 2, 50, generator=gen).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wo = w.clone()
    lens = torch.tensor([51, -1, 70], dtype=torch.int32).cuda()  # past weights, negative, past the table
    n, kept = fd.evict_kv(gk, gv, bt, lens, w, 20, weights_out=wo, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.FD_DEV_CAPACITY
    assert n.tolist() == lens.tolist() and (kept == -1).all() and torch.equal(wo, w)
    assert torch.equal(gk.cpu(), kp) and torch.equal(gv.cpu(), kp)
    # a page out of range: flagged, its rows skipped, the others moved
    status.zero_()
    bad = bt.clone()
    bad[0, 1] = 12
    bad[1, 1] = -1
    lens = torch.tensor([40, 40, 40], dtype=torch.int32).cuda()
    n, kept = fd.evict_kv(gk, gv, bad, lens, w, 20, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.FD_DEV_BAD_PAGE and n.tolist() == [20, 20, 20]
    k = kept[2, 0].cpu()
    j = torch.arange(20)
    assert torch.equal(gk.cpu()[8 + j // 16, j % 16, 0], kp[8 + k // 16, k % 16, 0])


def test_graph_replay_and_other_stream(fdlib):
    gen = torch.Generator().manual_seed(2)
    lens = torch.tensor([300, 90], dtype=torch.int32).cuda()
    bt, pages, spare = R.make_table(gen, [300, 90], 16, extra=40)
    kp, _ = R.make_pool(gen, pages, 16, 2, 64, torch.bfloat16)
    vp, _ = R.make_pool(gen, pages, 16, 2, 64, torch.bfloat16)
    dst = torch.full_like(bt, -1)
    dst[0, :7], dst[1, :6] = spare[:7], spare[7:13]
    w = torch.rand(2, 2, 300, generator=gen).cuda()
    a, b = [kp.cuda(), vp.cuda()], [kp.cuda(), vp.cuda()]
    bt, dst = bt.cuda(), dst.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n1, k1 = fd.evict_kv(*a, bt, lens, w, 100, 4, 20, dst_table=dst, stream=side)
    side.synchronize()
    fd.evict_kv(*b, bt, lens, w, 100, 4, 20, dst_table=dst)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n2, k2 = fd.evict_kv(*b, bt, lens, w, 100, 4, 20, dst_table=dst)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n1, n2) and torch.equal(k1, k2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replay_of_long_rows(fdlib):
    """Rows that a cluster of CTAs selects, captured and replayed on other weights."""
    gen = torch.Generator().manual_seed(4)
    L, ps, budget = 40000, 64, 20000
    bt, pages, spare = R.make_table(gen, [L], ps, extra=400)
    kp, _ = R.make_pool(gen, pages, ps, 1, 64, torch.bfloat16)
    dst = torch.full_like(bt, -1)
    dst[0, :313] = spare[:313]
    gk, gv, bt, dst = kp.cuda(), kp.cuda().clone(), bt.cuda(), dst.cuda()
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    w = torch.zeros(1, 1, L, device="cuda")
    call = lambda: fd.evict_kv(gk, gv, bt, lens, w, budget, 4, 1000, dst_table=dst)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, kept = call()
    for seed in range(3):
        v = torch.rand(1, 1, L, generator=torch.Generator().manual_seed(seed))
        w.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        keep = R.evict(v[0, 0], L, budget, 4, 1000)
        assert n.tolist() == [budget] and kept[0, 0].tolist() == keep.tolist()
        j = torch.arange(budget)
        old = kp[bt.cpu()[0, keep // ps].long(), keep % ps, 0]
        assert torch.equal(gk.cpu()[dst.cpu()[0, j // ps].long(), j % ps, 0], old)

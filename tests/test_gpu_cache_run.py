"""The cache operators as a serving loop uses them: prompts enter the cache
(append_kv_norm), every step appends a token, decodes and adds to the totals
(decode_weights), and sequences that pass their budget are cut back (evict_kv),
in place; against the same loop in float64 with the stored values.  And the
same with differential attention reading the cache."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests import cache_ref as R
from tests.test_gpu_append_norm import tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,diff", [("bf16", False), ("e4m3", False), ("bf16", True), ("f16", False)])
def test_serving_loop(fdlib, kv, diff):
    B, Hq, Hkv, D, ps, steps = 3, 8, 2, 128, 16, 12
    budget, sinks, recent = 48, 2, 12
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[kv]
    act = torch.float16 if kv == "f16" else torch.bfloat16
    gen = torch.Generator().manual_seed(11)
    prompts = [40, 7, 47]
    room = 64  # tokens of pages each sequence owns
    bt = torch.randperm(B * room // ps, generator=gen).to(torch.int32).view(B, -1)
    pages = bt.numel()
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, dt)
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, dt)
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    kp, vp, ks, vs, bt = g(kp), g(vp), g(ks), g(vs), g(bt)
    cos, sin = (t.cuda() for t in tables(256, D // 2))
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=gen)).to(act).cuda() for _ in range(2))
    lam = torch.rand(Hq, generator=gen).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, pos = i32([0] * B), i32([0] * B)
    totals = torch.zeros(B, Hkv, room, device="cuda")
    prob = fd.make_problem(B, Hq, Hkv, D, ps, room // ps, pages, act, dt)
    dec = fd.PagedDecoder(prob, [room] * B, track_weights=True)
    dif = fd.DiffDecoder(prob, [room] * B)
    common = dict(q_weight=qw, k_weight=kw, rotary_cos=cos, rotary_sin=sin, k_scale=ks, v_scale=vs)
    sc = dict(k_scale=ks, v_scale=vs)
    # the reference: stored K, V and totals of every (sequence, KV head), with bounds
    # on the totals' error; K and V are read back from the cache, which the append's
    # own tests hold to the formula
    held = [[[] for _ in range(Hkv)] for _ in range(B)]  # positions of the tokens kept, in order
    tot = [[torch.zeros(0, dtype=torch.float64) for _ in range(Hkv)] for _ in range(B)]

    def stored(b, h, n):
        at = torch.arange(n, device="cuda")
        pg, sl = bt[b, at // ps].long(), at % ps
        k, v = (p.view(torch.uint8)[pg, sl, h].view(dt) if kv == "e4m3" else p[pg, sl, h] for p in (kp, vp))
        k, v = k.float().double(), v.float().double()
        if kv == "e4m3":
            k, v = k * ks[pg, h].double()[:, None], v * vs[pg, h].double()[:, None]
        return k.cpu(), v.cpu()

    def take(T, new):
        qkv = torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=gen).to(act).cuda()
        q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
        out = fd.append_kv_norm(q, k, v, kp, vp, bt, lens, positions=pos, new_lens=i32(new), **common)
        for b in range(B):
            for h in range(Hkv):
                first = int(pos[b])
                held[b][h] += list(range(first, first + new[b]))
                tot[b][h] = torch.cat([tot[b][h], torch.zeros(new[b], dtype=torch.float64)])
        lens.add_(i32(new))
        pos.add_(i32(new))
        return out

    take(max(prompts), prompts)
    evicted = 0
    for step in range(steps):
        q = take(1, [1] * B)[:, 0].contiguous()
        if diff:
            out, _ = dif(q, kp, vp, bt, lens, lam, out_scale=1.0, **sc)
        _, _, _ = dec.decode_weights(q, kp, vp, bt, lens, totals, **sc)
        torch.cuda.synchronize()
        for b in range(B):
            L = int(lens[b])
            for h in range(Hkv):
                k, v = stored(b, h, L)
                qh = q[b, h * 4:h * 4 + 4].cpu().float().double()
                p = torch.softmax(qh @ k.T / D ** 0.5, -1)
                tot[b][h] += p.sum(0)
                # scores of norm about 1 * 11 are off by less than 2^-14; 12 steps and evictions add up
                assert torch.allclose(totals[b, h, :L].cpu().double(), tot[b][h], rtol=2.0 ** -10, atol=1e-6)
                if diff:
                    d = D // 2
                    o = [torch.softmax(qh[:, x] @ k[:, x].T / d ** 0.5, -1) @ v for x in (slice(0, d), slice(d, D))]
                    ref = o[0] - lam[h * 4:h * 4 + 4].cpu().double()[:, None] * o[1]
                    got = out[b, h * 4:h * 4 + 4].cpu().double()
                    # two outputs within 2^-10 of |V| <= 6 each, then bf16's rounding
                    assert ((got - ref).abs() <= 2 * 6 * 2.0 ** -10 + R.rounding(ref, act)).all()
        if int(lens.max()) > budget + 3:
            before = [[stored(b, h, int(lens[b])) for h in range(Hkv)] for b in range(B)]
            w = totals.cpu()
            n, kept = fd.evict_kv(kp, vp, bt, lens, totals, budget, sinks, recent, weights_out=totals, **sc)
            torch.cuda.synchronize()
            for b in range(B):
                L = int(lens[b])
                evicted += L - int(n[b])
                for h in range(Hkv):
                    keep = R.evict(w[b, h], L, budget, sinks, recent)
                    assert kept[b, h, :len(keep)].tolist() == keep.tolist()
                    held[b][h] = [held[b][h][i] for i in keep.tolist()]
                    tot[b][h] = tot[b][h][keep]
                    k, v = stored(b, h, len(keep))
                    # E4M3 codes may have been rounded again for another page's scale
                    tol = 2.0 ** -4 if kv == "e4m3" else 0.0
                    for now, was in ((k, before[b][h][0][keep]), (v, before[b][h][1][keep])):
                        assert ((now - was).abs() <= tol * was.abs() + (2.0 ** -8 if tol else 0.0)).all()
            lens.copy_(n)
    assert evicted > 0
    dec.check()
    dif.check()
    # what stays of every head: the first tokens and the latest ones among them, in order
    for b in range(B):
        for h in range(Hkv):
            assert held[b][h] == sorted(held[b][h]) and held[b][h][:sinks] == list(range(sinks))
            assert held[b][h][-recent:] == list(range(int(pos[b]) - recent, int(pos[b])))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_back_to_back_calls_equal_waited_ones(fdlib, kv):
    """Kernels that start while the one before drains: the same results, bit for
    bit, as with a synchronisation after every call."""
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kv]
    B, Hq, Hkv, D, ps, room, budget = 24, 16, 4, 128, 16, 2304, 1500
    res = []
    for wait in (True, False):
        gen = torch.Generator().manual_seed(5)
        dev = torch.Generator(device="cuda").manual_seed(6)
        bt = torch.randperm(B * room // ps, generator=gen).to(torch.int32).view(B, -1).cuda()
        kp, ks = R.make_pool(gen, bt.numel(), ps, Hkv, D, dt)
        vp, vs = R.make_pool(gen, bt.numel(), ps, Hkv, D, dt)
        kp, vp, ks, vs = (None if t is None else t.cuda() for t in (kp, vp, ks, vs))
        sc = dict(k_scale=ks, v_scale=vs)
        cos, sin = (t.cuda() for t in tables(6000, D // 2))
        w, lam = torch.ones(D, dtype=torch.bfloat16, device="cuda"), torch.rand(Hq, generator=dev, device="cuda")
        lens = torch.randint(1400, 1900, (B,), generator=dev, device="cuda", dtype=torch.int32)
        pos = lens.clone()
        prob = fd.make_problem(B, Hq, Hkv, D, ps, room // ps, bt.numel(), torch.bfloat16, dt)
        dec, dif = fd.PagedDecoder(prob, [1900] * B, track_weights=True), fd.DiffDecoder(prob, [1900] * B)
        totals = torch.zeros(B, Hkv, room, device="cuda")
        feed = [torch.randn(B, 7, (Hq + 2 * Hkv) * D, generator=dev, device="cuda").bfloat16() for _ in range(6)]
        outs = []
        step = torch.cuda.synchronize if wait else (lambda: None)
        torch.cuda.synchronize()
        for x in feed:
            q, k, v = (t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))
            q = fd.append_kv_norm(q, k, v, kp, vp, bt, lens, q_weight=w, k_weight=w, rotary_cos=cos, rotary_sin=sin,
                                  positions=pos, **sc)
            step()
            lens, pos = lens + 7, pos + 7
            last = q[:, -1].contiguous()
            out, lse, _ = dec.decode_weights(last, kp, vp, bt, lens, totals, **sc)
            step()
            out2, lse2 = dif(last, kp, vp, bt, lens, lam, norm_weight=w, **sc)
            step()
            lens, kept = fd.evict_kv(kp, vp, bt, lens, totals, budget, 4, 200, weights_out=totals, **sc)
            step()
            outs += [q, out, lse, out2, lse2, lens, kept]
        torch.cuda.synchronize()
        dec.check()
        dif.check()
        res.append(outs + [totals, kp.view(torch.uint8), vp.view(torch.uint8)])
    assert all(torch.equal(a, b) for a, b in zip(*res))

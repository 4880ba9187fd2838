"""Cross attention and decode behind shared prefixes as a serving program uses
them: after the appends that fill the pages, in captured graphs, on other
streams, one call behind the other, with many KV rows and groups, over pools
past 2^31 elements, both ways of marshalling, and when a device-side wait runs
out."""
import ctypes
import random

import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests import cache_ref as R
from tests.shared_ref import Cross, Prefix

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


def cross_decoder(c, d, **opts):
    return fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, beams=c.beams, **opts)


def prefix_decoder(c, d, **opts):
    return fd.PrefixDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["prefix_table"], c.plens, c.of,
                                      d["block_table"], c.lens, **opts)


@pytest.mark.parametrize("kv,q", [(BF16, BF16), (E4M3, F16)], ids=["bf16", "e4m3-f16"])
def test_many_kv_rows(fdlib, kv, q):
    """More KV rows than a warp has lanes: lengths from 0 in no order, counts
    of queries among them."""
    rng = random.Random(1)
    lens = [rng.choice([0, 1, 17, 128, 200, 333]) for _ in range(70)]
    counts = [rng.randint(0, 20) for _ in lens]
    for q_lens, beams in ((None, 1), (counts, 1), ([x % 4 for x in range(140)], 2)):
        T = 20 if beams == 1 else 3
        c = Cross(2, lens, beams=beams, T=T, Hq=4, Hkv=2, D=64, kv=kv, q=q, q_lens=q_lens)
        d = c.device()
        for splits in (0, 2):
            dec = cross_decoder(c, d, num_splits=splits)
            out, lse = torch.full_like(d["q"], 7.0), torch.full(d["q"].shape[:-1], 7.0, device="cuda")
            dec(**d, out=out, lse=lse)
            dec.check()
            c.verify(out, lse, untouched=7.0, what="many rows")


@pytest.mark.parametrize("kv,q", [(BF16, BF16), (F16, F16), (E4M3, BF16)], ids=["bf16", "f16", "e4m3"])
def test_many_groups(fdlib, kv, q):
    """90 prefixes, most with one or two sequences, some with none."""
    rng = random.Random(2)
    of = [rng.randint(-1, 89) for _ in range(120)]
    c = Prefix(3, [rng.randint(0, 300) for _ in range(90)], of, [rng.randint(1, 40) for _ in of], Hq=6, Hkv=2, D=64, kv=kv, q=q)
    d = c.device()
    for splits in (0, 2):
        dec = prefix_decoder(c, d, num_splits=splits)
        out, lse = dec(**d)
        dec.check()
        c.verify(out, lse, what="many groups")
    ref = out
    # offsets that fall: cut where they do, the groups before that are right
    bad = dec.offsets.clone()
    bad[40] = 0
    good = dec.members[:int(bad[39])].long()
    dec.offsets.copy_(bad)
    out, _ = dec(**d)
    with pytest.raises(fd.FdError) as e:
        dec.check()
    assert e.value.code == _lib.FD_ERR_BAD_PAGE
    assert torch.equal(out[good], ref[good])


@pytest.mark.parametrize("seed", range(24))
def test_drawn_cases(fdlib, seed):
    rng = random.Random(seed)
    kv = rng.choice([F16, BF16, E4M3])
    q = rng.choice([F16, BF16]) if kv == E4M3 else kv
    kw = dict(Hkv=rng.choice([1, 2, 3]), D=rng.choice([64, 128]), ps=rng.choice([16, 32, 48, 64, 112, 128]), kv=kv, q=q)
    kw["Hq"] = kw["Hkv"] * rng.choice([1, 2, 3, 5, 8, 12])
    if rng.random() < 0.5:
        beams, T = rng.choice([1, 1, 2, 5]), rng.choice([1, 2, 30, 150])
        lens = [rng.choice([0, rng.randint(1, 1200)]) for _ in range(rng.randint(1, 5))]
        q_lens = [rng.randint(0, T) for _ in range(len(lens) * beams)] if rng.random() < 0.5 else None
        c = Cross(seed, lens, beams=beams, T=T, q_lens=q_lens, **kw)
        d = c.device()
        dec = cross_decoder(c, d, num_splits=rng.choice([0, 0, 3]))
        out, lse = torch.full_like(d["q"], 7.0), torch.full(d["q"].shape[:-1], 7.0, device="cuda")
        dec(**d, out=out, lse=lse)
        dec.check()
        c.verify(out, lse, untouched=7.0, what=f"seed {seed}")
    else:
        T, P = rng.choice([1, 1, 2, 5]), rng.randint(1, 4)
        of = [rng.randint(-1, P - 1) for _ in range(rng.randint(1, 40))]
        c = Prefix(seed, [rng.randint(0, 900) for _ in range(P)], of, [rng.randint(T, 200) for _ in of], T=T, **kw)
        d = c.device()
        dec = prefix_decoder(c, d, num_splits=rng.choice([0, 0, 3]))
        out, lse = dec(**d)
        dec.check()
        c.verify(out, lse, what=f"seed {seed}")


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_encoder_states_appended_then_attended(fdlib, kv):
    """The states of two inputs written by append_kv_norm (no queries, no
    rotation), then three layers' worth of prompt and single-token calls."""
    c = Cross(4, [75, 130], T=12, Hq=4, Hkv=2, D=64, kv=kv, ps=16)
    d = c.device()
    n = torch.tensor(c.kv_lens, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(5)
    kn, vn = (torch.randn((2, 130, 2, 64), generator=gen).to(BF16) for _ in "kv")
    if kv == E4M3:  # scales with room, NaN nowhere
        c.ks, c.vs = (torch.full_like(s, 0.02) for s in (c.ks, c.vs))
        d["k_scale"], d["v_scale"] = c.ks.cuda(), c.vs.cuda()
    fd.append_kv_norm(None, kn.cuda(), vn.cuda(), d["k_pages"], d["v_pages"], d["block_table"], torch.zeros_like(n),
                      new_lens=n, k_scale=d["k_scale"], v_scale=d["v_scale"])
    c.k, c.v = d["k_pages"].cpu(), d["v_pages"].cpu()
    prompt = cross_decoder(c, d)
    out, lse = prompt(**d)
    prompt.check()
    c.verify(out, lse, what="prompt")
    one = Cross(4, [75, 130], T=1, Hq=4, Hkv=2, D=64, kv=kv, ps=16)
    one.k, one.v, one.ks, one.vs, one.table = c.k, c.v, c.ks, c.vs, c.table
    q1 = one.q[:, 0].contiguous().cuda()
    step = fd.CrossDecoder.for_pools(q1, d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens)
    out, lse = step(q1, *(d[k] for k in ("k_pages", "v_pages", "block_table", "kv_lens")), k_scale=d["k_scale"],
                    v_scale=d["v_scale"])
    step.check()
    one.verify(out[:, None], lse[:, None], what="step")


def test_prefix_steps_agree_with_whole_sequences(fdlib):
    """Several decode steps behind page-aligned prefixes, each token appended
    first: PrefixDecoder against PagedDecoder over prefix and own pages together."""
    c = Prefix(6, [64, 160], [1, 0, 1, -1, 0], [3, 17, 30, 9, 1], Hq=8, Hkv=2, D=128)
    d = c.device()
    ps, room = 16, 64
    gen = torch.Generator().manual_seed(7)
    pages = d["k_pages"].shape[0] + 20
    kp = torch.zeros((pages, ps, 2, 128), dtype=BF16, device="cuda")
    vp = torch.zeros_like(kp)
    kp[:pages - 20], vp[:pages - 20] = d["k_pages"], d["v_pages"]
    own = torch.arange(pages - 20, pages, dtype=torch.int32).view(5, 4)
    for b, L in enumerate(c.lens):  # the own tokens move to pages with room
        for j in range(-(-L // ps)):
            kp[int(own[b, j])], vp[int(own[b, j])] = d["k_pages"][int(c.table[b, j])], d["v_pages"][int(c.table[b, j])]
    lens = list(c.lens)
    whole, full = [], []
    for b, p in enumerate(c.of):
        pre = c.ptable[p, :c.plens[p] // ps].tolist() if p >= 0 else []
        whole.append(pre + own[b].tolist())
        full.append(16 * len(pre))
    cols = max(map(len, whole))
    whole = torch.tensor([w + [-1] * (cols - len(w)) for w in whole], dtype=torch.int32).cuda()
    q0 = torch.zeros(5, 8, 128, dtype=BF16, device="cuda")
    dec = fd.PrefixDecoder.for_pools(q0, kp, vp, d["prefix_table"], c.plens, c.of, own.cuda(), lens, max_seq_len=room)
    ref = fd.PagedDecoder.for_pools(q0, kp, vp, whole, [f + n for f, n in zip(full, lens)], max_seq_len=cols * ps)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    off = torch.tensor(full, dtype=torch.int32, device="cuda")
    for step in range(20):
        q, k, v = (torch.randn(5, h, 128, generator=gen).to(BF16).cuda() for h in (8, 2, 2))
        fd.append_kv(BF16, k, v, kp, vp, own.cuda(), sl)
        sl = sl + 1
        out, lse = dec(q, kp, vp, d["prefix_table"], d["prefix_lens"], own.cuda(), sl)
        want, wlse = ref(q, kp, vp, whole, off + sl)
        dec.check()
        ref.check()
        # both are within r_p sum p |v| of the exact result and rounded to bf16: 2^-8 each, |v| below 5
        assert float((out.float() - want.float()).abs().max()) <= 5 * (2.0 ** -8 + 2.0 ** -7)
        assert float((lse - wlse).abs().max()) <= 2.0 ** -12  # scores of up to 2^5, each off by 2^-19 of that, and sums


def test_captured_and_replayed(fdlib):
    """Calls in one CUDA graph, replayed with other queries, lengths and groups."""
    c = Cross(8, [400, 90, 700], T=40, Hq=8, Hkv=2, D=64, kv=BF16)
    p = Prefix(9, [200, 50], [0, 1, 0, -1], [9, 20, 3, 40], Hq=8, Hkv=2, D=64, kv=BF16)
    cd, pd = c.device(), p.device()
    cdec, pdec = cross_decoder(c, cd, num_splits=3), prefix_decoder(p, pd, num_splits=2)
    counts = torch.tensor([40, 3, 17], dtype=torch.int32, device="cuda")
    cd["q_lens"] = counts
    co, cl = torch.empty_like(cd["q"]), torch.empty(cd["q"].shape[:-1], device="cuda")
    po, pl = torch.empty_like(pd["q"]), torch.empty(pd["q"].shape[:-1], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            cdec(**cd, out=co, lse=cl)
            pdec(**pd, out=po, lse=pl)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cdec(**cd, out=co, lse=cl)
        pdec(**pd, out=po, lse=pl)
        cdec(**cd, out=co, lse=cl)
    for step in range(3):
        c.q, p.q = c.q.roll(1, 0), p.q.roll(1, 0)
        cd["q"].copy_(c.q)
        pd["q"].copy_(p.q[:, 0])
        c.kv_lens = [400 - 50 * step, 90, 700 - 300 * step]
        cd["kv_lens"].copy_(torch.tensor(c.kv_lens, dtype=torch.int32))
        c.q_lens = [40 - step, 3 + step, 17]
        counts.copy_(torch.tensor(c.q_lens, dtype=torch.int32))
        p.of = [(o + step) % 3 - 1 for o in (1, 2, 0, 2)]
        pdec.regroup(p.of)
        co.fill_(7.0)
        cl.fill_(7.0)
        g.replay()
        cdec.check()
        pdec.check()
        c.verify(co, cl, untouched=7.0, what=f"replay {step}")
        p.verify(po, pl, what=f"replay {step}")


def test_calls_behind_one_another_and_on_other_streams(fdlib):
    """A hundred calls without a wait between them give what each gives alone;
    two decoders on two streams do not meet."""
    c = Cross(10, [300, 700, 20], T=30, Hq=4, Hkv=2, D=128, kv=BF16)
    p = Prefix(11, [300], [0] * 20, [5 + i for i in range(20)], Hq=8, Hkv=2, D=128, kv=BF16)
    cd, pd = c.device(), p.device()
    c1, c2 = cross_decoder(c, cd, num_splits=2), cross_decoder(c, cd)
    p1 = prefix_decoder(p, pd, num_splits=2)
    want, _ = c1(**cd)
    want2, _ = c2(**cd)
    pw, _ = p1(**pd)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for i in range(100):
        with torch.cuda.stream(s1):
            a, _ = c1(**cd)
            b, _ = p1(**pd)
        e, _ = c2(**cd, stream=s2)
        if i % 10 == 9:
            got.append((a, b, e))
    torch.cuda.synchronize()
    for dec in (c1, c2, p1):
        dec.check()
    for a, b, e in got:
        assert torch.equal(a, want) and torch.equal(b, pw) and torch.equal(e, want2)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_far_pages(fdlib, kv):
    """Pages at the far end of a pool past 2^31 elements (2^32 bytes) give bit
    for bit what the same pages of a small one give."""
    far = 140000 if kv == BF16 else 270000  # of 128 x 128 elements
    c = Cross(12, [300, 900], T=40, Hq=4, Hkv=1, D=128, kv=kv, ps=128)
    p = Prefix(13, [500], [0, 0, -1], [90, 3, 200], Hq=4, Hkv=1, D=128, kv=kv, ps=128)
    res = []
    for base in (0, far):
        row = []
        for x in (c, p):
            d = x.device()
            for name in ("k_pages", "v_pages"):
                small = d[name]
                big = torch.empty((small.shape[0] + base,) + small.shape[1:], dtype=kv, device="cuda")
                big.view(torch.uint8)[base:] = small.view(torch.uint8)
                d[name] = big
            for name in ("k_scale", "v_scale"):
                if d[name] is not None:
                    s = torch.ones((d[name].shape[0] + base, 1), device="cuda")
                    s[base:] = d[name]
                    d[name] = s
            for name in ("block_table", "prefix_table"):
                if name in d:
                    d[name] = torch.where(d[name] >= 0, d[name] + base, d[name])
            dec = cross_decoder(c, d) if x is c else prefix_decoder(p, d)
            out, lse = dec(**d)
            dec.check()
            row += [out, lse]
            del d, big
            torch.cuda.empty_cache()
        res.append(row)
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("T", [1, 30])
def test_both_ways_of_marshalling(fdlib, monkeypatch, T):
    c = Cross(14, [300, 70], T=T, Hq=4, Hkv=2, D=64, beams=2, kv=E4M3)
    p = Prefix(15, [130, 40], [0, 1, -1, 0], [9, 20, 3, 40], T=min(T, 3), Hq=8, Hkv=2, D=64, kv=F16)
    cd, pd = c.device(), p.device()
    cdec, pdec = cross_decoder(c, cd), prefix_decoder(p, pd)
    counts = torch.full((4,), T, dtype=torch.int32, device="cuda")
    res = []
    for native in (True, False):
        if native:
            assert _lib.fast()
        else:
            monkeypatch.setattr(_lib, "_fast", False)
        a = cdec(**cd)
        b = cdec(**{**cd, "q_lens": counts}, out=torch.empty_like(cd["q"]), lse=a[1].clone())
        e = cdec(**cd, want_lse=False)
        assert e[1] is None
        f = pdec(**pd)
        g = pdec(**pd, out=torch.empty_like(pd["q"]), want_lse=False)
        assert g[1] is None
        res.append([*a, *b, e[0], *f, g[0]])
        cdec.check()
        pdec.check()
    assert all(torch.equal(x, y) for x, y in zip(*res))


@pytest.mark.parametrize("status", ["FD_ERR_CUDA", "FD_ERR_INVALID_ARG"])
def test_failed_and_refused_calls(fdlib, monkeypatch, status):
    """A call whose launches failed raises and is not made again; a refused one
    goes the Python way.  The entry points are stand-ins that launch nothing."""
    c = Cross(18, [30], T=2, Hq=4, Hkv=2, D=64)
    p = Prefix(19, [40], [0, 0], [9, 20], Hq=4, Hkv=2, D=64)
    cd, pd = c.device(), p.device()
    cdec, pdec = cross_decoder(c, cd), prefix_decoder(p, pd)
    fast = _lib.fast()
    assert fast
    names = ("fd_cross_paged", "fd_decode_paged_prefix")
    real = [ctypes.cast(getattr(fdlib, n), ctypes.c_void_p).value for n in names]
    code, calls, again = getattr(_lib, status), [], []

    @ctypes.CFUNCTYPE(ctypes.c_int)
    def stub():
        calls.append(code)
        return code

    fast.init_shared(*[ctypes.cast(stub, ctypes.c_void_p).value] * 2)
    try:
        for n in names:
            monkeypatch.setattr(_lib, n, lambda *a, **kw: again.append(a))
        for i, f in enumerate((lambda: cdec(**cd), lambda: pdec(**pd))):
            if code == _lib.FD_ERR_CUDA:
                with pytest.raises(fd.FdError) as e:
                    f()
                assert e.value.code == code and "fd_" in str(e.value) and not again
            else:
                f()
                assert len(again) == i + 1
            assert len(calls) == i + 1
    finally:
        fast.init_shared(*real)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_wait_limits(fdlib, kv):
    """Loads that start later than the wait limit: the status says so, check()
    clears the workspace, and a plan without the hook then gives right results
    on it."""
    c = Cross(16, [900, 300], T=60, Hq=4, Hkv=2, D=64, kv=kv)
    d = c.device()
    late = cross_decoder(c, d, timeout_us=200, debug_stall_us=20000)
    late(**d)
    torch.cuda.synchronize()
    assert int(late.status.item()) & _lib.FD_DEV_TIMEOUT
    with pytest.raises(fd.FdError) as e:
        late.check()
    assert e.value.code == _lib.FD_ERR_TIMEOUT
    late.plan.debug_stall_us = 0
    late.plan.timeout_us = 5000
    for _ in range(2):
        out, lse = late(**d)
        late.check()
        c.verify(out, lse, what="after a timeout")
    p = Prefix(17, [400], [0, 0, 0], [9, 20, 3], Hq=4, Hkv=2, D=64, kv=kv)
    d = p.device()
    dec = prefix_decoder(p, d, timeout_us=200, prefix_stall_us=20000)
    dec(**d)
    with pytest.raises(fd.FdError) as e:
        dec.check()
    assert e.value.code == _lib.FD_ERR_TIMEOUT
    dec.plan.shared.debug_stall_us = 0
    dec.plan.shared.timeout_us = 5000
    out, lse = dec(**d)
    dec.check()
    p.verify(out, lse, what="after a timeout")

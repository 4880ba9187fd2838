"""The native marshalling of the cache operators (csrc/torch_binding.cpp) and the
Python binding make the same calls: equal results on the same inputs, for every
operator, and every call that is not the ordinary case goes the Python way."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests import cache_ref as R
from tests.test_gpu_weights import setup

pytestmark = pytest.mark.gpu


@pytest.fixture
def python_way(monkeypatch):
    def off():
        monkeypatch.setattr(_lib, "_fast", False)
    return off


def test_the_binding_is_built_and_takes_ordinary_calls(fdlib):
    fast = _lib.fast()
    assert fast
    q, kp, vp, _, _, bt = (None if t is None else t.cuda() for t in setup("bf16", "bf16", [40, 9], 8, 2, 64, 16))
    dl = torch.tensor([40, 9], dtype=torch.int32).cuda()
    w = torch.rand(2, 2, 64).cuda()
    assert fast.evict_kv(kp, vp, bt, dl, w, 20, 2, 3, None, None, None, None, None) is not None
    # other types, shapes, layouts and places are handed back
    for bad in ((kp, vp, bt, dl, w.half(), 20, 2, 3), (kp, vp, bt.long(), dl, w, 20, 2, 3), (kp, vp, bt, dl, w.cpu(), 20, 2, 3),
                (kp, vp[:-1], bt, dl, w, 20, 2, 3), (kp, vp, bt, dl, w.transpose(0, 1), 20, 2, 3), (kp, vp, bt, dl, w, 0, 0, 0),
                (kp, vp, bt, dl, w, 20, 15, 6), (kp, vp, bt, dl, None, 20, 2, 3), (kp, vp, bt, dl, w, "20", 2, 3),
                (kp, vp, bt, dl, w, 1 << 40, 2, 3)):
        assert fast.evict_kv(*bad, None, None, None, None, None) is None
    assert fast.evict_kv(kp) is None
    torch.cuda.synchronize()


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
def test_append_both_ways(fdlib, python_way, kv):
    lens = [0, 20, 33]
    act = torch.float16 if kv == "f16" else torch.bfloat16
    res = []
    for native in (True, False):
        if not native:
            python_way()
        gen = torch.Generator().manual_seed(1)
        bt, pages, _ = R.make_table(gen, [n + 3 for n in lens], 16)
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[kv]
        kp, ks = R.make_pool(gen, pages, 16, 2, 64, dt)
        vp, vs = R.make_pool(gen, pages, 16, 2, 64, dt)
        g = lambda t: None if t is None else t.cuda()  # noqa: E731
        gk, gv = g(kp), g(vp)
        rows = torch.randn(3, 3, 12 * 64, generator=gen).to(act).cuda()
        q, k, v = (x.unflatten(-1, (-1, 64)) for x in rows.split([8 * 64, 2 * 64, 2 * 64], -1))
        w = torch.randn(64, generator=gen).cuda()
        cos, sin = torch.randn(40, 32, generator=gen).cuda(), torch.randn(40, 32, generator=gen).cuda()
        kw = dict(q_weight=w, k_weight=w, rotary_cos=cos, rotary_sin=sin, k_scale=g(ks), v_scale=g(vs),
                  new_lens=torch.tensor([3, 2, 3], dtype=torch.int32).cuda())
        dl = torch.tensor(lens, dtype=torch.int32).cuda()
        out = fd.append_kv_norm(q, k, v, gk, gv, bt.cuda(), dl, q_out=q, **kw)
        assert out is q
        new = fd.append_kv_norm(q, k, v, gk, gv, bt.cuda(), dl, **kw)
        only = fd.append_kv_norm(None, k[:, 0], v[:, 0], gk, gv, bt.cuda(), dl, k_scale=g(ks), v_scale=g(vs))
        assert only is None
        new[1, 2] = 0  # not written: beyond its sequence's new tokens
        res.append([out.clone(), new, gk.view(torch.uint8).clone(), gv.view(torch.uint8).clone()])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("kv,q_len", [("bf16", 1), ("f16", 3), ("e4m3", 1)])
def test_decoders_both_ways(fdlib, python_way, kv, q_len):
    lens = [700, 33, q_len]
    act = "f16" if kv == "f16" else "bf16"
    q, kp, vp, ks, vs, bt = (None if t is None else t.cuda() for t in setup(kv, act, lens, 8, 2, 128, 16, q_len))
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    lam, nw = torch.rand(8).cuda(), torch.rand(128).cuda()
    sc = dict(k_scale=ks, v_scale=vs)
    dec = fd.PagedDecoder.for_pools(q, kp, vp, bt, lens, track_weights=True, num_splits=1)
    dif = fd.DiffDecoder.for_pools(q, kp, vp, bt, lens, num_splits=1)
    res = []
    for native in (True, False):
        if not native:
            python_way()
        w = torch.zeros(3, 2, 700, device="cuda")
        o1, l1, t1 = dec.decode_weights(q, kp, vp, bt, dl, w, **sc)
        assert t1 is w
        o2, l2, t2 = dec.decode_weights(q, kp, vp, bt, dl, None, weights_out=torch.zeros_like(w), out=torch.empty_like(q),
                                        want_lse=False, **sc)
        assert l2 is None
        o3, l3 = dif(q, kp, vp, bt, dl, lam, norm_weight=nw, out_scale=2, **sc)
        o4, l4 = dif(q, kp, vp, bt, dl, lam, out=torch.empty_like(q), lse=l3.clone(), **sc)
        res.append([o1, l1, t1, o2, t2, o3, l3, o4, l4])
        dec.check()
        dif.check()
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_evict_both_ways(fdlib, python_way):
    gen = torch.Generator().manual_seed(1)
    lens = [300, 40]
    bt, pages, _ = R.make_table(gen, lens, 16)
    kp, _ = R.make_pool(gen, pages, 16, 2, 64, torch.bfloat16)
    w = torch.rand(2, 2, 300, generator=gen).cuda()
    res = []
    for native in (True, False):
        if not native:
            python_way()
        gk, gv, wo = kp.cuda(), kp.cuda().clone(), torch.zeros_like(w)
        n, kept = fd.evict_kv(gk, gv, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), w, 100, 4, 20, weights_out=wo)
        res.append([n, kept, gk, gv, wo])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))

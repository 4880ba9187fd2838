"""The cache operators on pools past 2^31 elements and 2^32 bytes: pages at the
far end of a large pool give bit for bit what the same pages of a small one give."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_far_pages(fdlib, kv):
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kv]
    B, Hq, Hkv, D, ps = 2, 4, 1, 128, 128
    far = 140000 if kv == "bf16" else 270000  # 2.3e9 elements of 2 bytes, 4.4e9 of 1
    gen = torch.Generator().manual_seed(1)
    lens = [300, 900]
    bt, pages, spare = R.make_table(gen, [n + 40 for n in lens], ps, extra=10, pad_cols=1)
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, dt)
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, dt)
    dst = torch.full_like(bt, -1)
    dst[0, :3], dst[1, :4] = spare[:3], spare[3:7]
    qkv = torch.randn(B, 40, (Hq + 2 * Hkv) * D, generator=gen).bfloat16().cuda()
    q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
    lam, w = torch.rand(Hq, generator=gen).cuda(), torch.ones(D).cuda()
    res = []
    for base in (0, far - pages):
        n = pages + base
        pools = []
        for p in (kp, vp):
            big = torch.empty((n, ps, Hkv, D), dtype=dt, device="cuda")
            big.view(torch.uint8)[base:] = p.view(torch.uint8).cuda()
            pools.append(big)
        sc = {}
        if ks is not None:
            for name, s in (("k_scale", ks), ("v_scale", vs)):
                sc[name] = torch.ones(n, Hkv, device="cuda")
                sc[name][base:] = s.cuda()
        table = torch.where(bt >= 0, bt + base, bt).cuda()
        to = torch.where(dst >= 0, dst + base, dst).cuda()
        dl = torch.tensor(lens, dtype=torch.int32).cuda()
        new_q = fd.append_kv_norm(q, k, v, *pools, table, dl, q_weight=w, k_weight=w, **sc)
        dl = dl + 40
        now = [n + 40 for n in lens]
        one = new_q[:, -1].contiguous()
        dec = fd.PagedDecoder.for_pools(one, *pools, table, now, track_weights=True)
        out, lse, totals = dec.decode_weights(one, *pools, table, dl, None, weights_out=torch.zeros(B, Hkv, 1000, device="cuda"),
                                              **sc)
        dif = fd.DiffDecoder.for_pools(one, *pools, table, now)
        out2, _ = dif(one, *pools, table, dl, lam, **sc)
        new_lens, kept = fd.evict_kv(*pools, table, dl, totals, 380, 4, 30, dst_table=to, **sc)
        same, _ = fd.evict_kv(*pools, table, dl, totals, 400, 4, 30, **sc)
        torch.cuda.synchronize()
        dec.check()
        dif.check()
        res.append([new_q, out, lse, totals, out2, new_lens, kept, same] + [p.view(torch.uint8)[base:].clone() for p in pools])
        del pools, sc
        torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(*res))

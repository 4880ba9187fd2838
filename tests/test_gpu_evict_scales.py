"""E4M3 codes that move between places of one scale stay as they are, whatever
that scale is: a page of zeros may have scale 0."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, 1e-42, float("inf")])
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_codes_stay_between_equal_scales(fdlib, D, fresh, scale):
    """Head 0 has `scale` on every page, head 1 an ordinary one."""
    ps, H, lens, budget, gen = 16, 2, [100, 40], 50, torch.Generator().manual_seed(D)
    bt, pages, spare = R.make_table(gen, lens, ps, extra=7)
    kp, ks = R.make_pool(gen, pages, ps, H, D, torch.float8_e4m3fn)
    vp, _ = R.make_pool(gen, pages, ps, H, D, torch.float8_e4m3fn)
    ks = torch.full_like(ks, 0.5)
    ks[:, 0] = scale
    dst = None
    if fresh:
        dst = torch.full_like(bt, -1)
        dst[0, :4], dst[1, :3] = spare[:4], spare[4:7]
    w = torch.rand(2, H, 100, generator=gen)
    gk, gv = kp.cuda(), vp.cuda()
    n, kept = fd.evict_kv(gk, gv, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), w.cuda(), budget, 2, 10,
                          dst_table=None if dst is None else dst.cuda(), k_scale=ks.cuda(), v_scale=ks.cuda())
    torch.cuda.synchronize()
    kept, to = kept.cpu(), bt if dst is None else dst
    for b in range(2):
        for h in range(H):
            src = kept[b, h, :int(n[b])].long()
            at = torch.arange(len(src))
            for old, new in ((kp, gk.cpu()), (vp, gv.cpu())):
                got = new.view(torch.uint8)[to[b, at // ps].long(), at % ps, h]
                assert torch.equal(got, old.view(torch.uint8)[bt[b, src // ps].long(), src % ps, h])

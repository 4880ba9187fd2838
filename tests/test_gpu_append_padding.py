"""What lies behind a sequence's new tokens in a padded append: neither read nor
written, whatever the size of the call.  Reads that would end behind the buffer
cannot be seen in a result, so here the padding holds NaN inside the buffer and
the call has to equal the one of the live tokens alone."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests import cache_ref as R
from tests.test_gpu_append_norm import bits, tables

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("T,live,Hq,Hkv,rd", [(8, 3, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 8, 2, 0), (5, 0, 3, 3, 34),
                                              (2500, 1700, 9, 3, 128)])
def test_padding_is_left_alone(fdlib, kv, act, T, live, Hq, Hkv, rd):
    D, ps, gen = 128, 16, torch.Generator().manual_seed(T)
    width = (Hq + 2 * Hkv) * D
    rows = torch.full((1, T, width), float("nan"), dtype=DT[act])
    rows[:, :live] = torch.randn(1, live, width, generator=gen).to(DT[act])
    bt, pages, _ = R.make_table(gen, [20 + T], ps)
    kp, ks = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    vp, vs = R.make_pool(gen, pages, ps, Hkv, D, DT[kv])
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    cos, sin = tables(20 + T, rd // 2) if rd else (None, None)
    w = (1 + 0.3 * torch.randn(D, generator=gen)).to(DT[act]).cuda()
    kw = dict(q_weight=w, k_weight=w, rotary_cos=g(cos), rotary_sin=g(sin), k_scale=g(ks), v_scale=g(vs))
    lens = torch.tensor([20], dtype=torch.int32).cuda()

    def call(x, **more):
        q, k, v = (t.unflatten(-1, (-1, D)) for t in x.cuda().split([Hq * D, Hkv * D, Hkv * D], -1))
        pools = [kp.cuda(), vp.cuda()]
        out = torch.full((1, x.shape[1], Hq, D), 7.0, dtype=DT[act], device="cuda")
        fd.append_kv_norm(q, k, v, *pools, bt.cuda(), lens, q_out=out, **kw, **more)
        return [out] + pools

    got = call(rows, new_lens=torch.tensor([live], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert (got[0][:, live:] == 7.0).all()
    want = call(rows[:, :live]) if live else [got[0], kp.cuda(), vp.cuda()]
    torch.cuda.synchronize()
    assert torch.equal(bits(got[0][:, :live]), bits(want[0][:, :live]))
    assert torch.equal(bits(got[1]), bits(want[1])) and torch.equal(bits(got[2]), bits(want[2]))

"""An infinite key element that hides its token from every query head of a KV
head (all scores -inf): its weight is 0, whatever the number of heads."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.test_gpu_weights import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "f16"])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 9])
@pytest.mark.parametrize("opts", [dict(num_splits=1), dict(num_splits=3), dict(q_len=2)])
def test_hidden_token_has_no_weight(fdlib, kv, G, opts):
    lens, Hkv, D, ps, q_len = [300, 40], 2, 64, 16, opts.get("q_len", 1)
    q, kp, vp, _, _, bt = setup(kv, kv, lens, G * Hkv, Hkv, D, ps, q_len, seed=G)
    q[..., 0] = -q[..., 0].abs() - 0.5
    hidden = [7, 33]
    for t in hidden:
        kp[bt[0, t // ps].long(), t % ps, :, 0] = float("inf")
    w = torch.zeros(2, Hkv, 300, device="cuda")
    dec = fd.PagedDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, track_weights=True, **opts)
    out, lse, w = dec.decode_weights(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), w)
    torch.cuda.synchronize()
    dec.check()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert (w[0, :, hidden] == 0).all()
    # the others share the weight: G * q_len rows, each to 2^-15 (300 of them)
    assert torch.allclose(w.double().sum(-1).cpu(), torch.full((2, Hkv), float(G * q_len), dtype=torch.float64), rtol=2e-4)


@pytest.mark.parametrize("kv", ["bf16", "f16"])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("opts", [dict(num_splits=1), dict(num_splits=3), dict(q_len=2)])
def test_key_hidden_from_one_map_is_seen_by_the_other(fdlib, kv, half, G, opts):
    """An infinite element in one half of a differential key: as a large finite one."""
    lens, Hkv, D, ps, q_len, dim = [300, 40], 2, 64, 16, opts.get("q_len", 1), half * 32
    q, kp, vp, _, _, bt = setup(kv, kv, lens, G * Hkv, Hkv, D, ps, q_len, seed=G)
    q[..., dim] = -q[..., dim].abs() - 0.5
    dec = fd.DiffDecoder.for_pools(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), lens, **opts)
    res = []
    for x in (float("inf"), 3e4):  # scores of -inf, and of less than -2000: weights of 0 either way
        for t in (7, 33):
            kp[bt[0, t // ps].long(), t % ps, :, dim] = x
        res.append(dec(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                       torch.full((G * Hkv,), 0.5).cuda(), norm_weight=torch.ones(D).cuda()))
    torch.cuda.synchronize()
    dec.check()
    for a, b in zip(*res):
        assert torch.isfinite(a).all() and torch.equal(a, b)

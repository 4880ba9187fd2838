"""Plans of decode_weights and differential attention go by the registers of the
kernel instances that run: two CTAs per SM only where two are resident.  The
rule for a host without a device and the device's own answer have to agree, so
the same expectations are checked on both."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib

E4M3, BF16, F16 = torch.float8_e4m3fn, torch.bfloat16, torch.float16


def plans(kv, act, B, L, Hq, Hkv, D, ps):
    blocks = -(-L // ps)
    p = _lib.make_problem(B, Hq, Hkv, D, ps, blocks, B * blocks, act, kv)
    return [f(p, [L] * B, num_sms=152) for f in (_lib.fd_plan, _lib.fd_plan_weights, _lib.fd_plan_diff)]


# shapes whose plain plan has two CTAs an SM: short items, small boxes, a small grid;
# and how many the score-writing and the differential instances leave room for
CASES = [(E4M3, BF16, 256, 1024, 32, 8, 128, 64, 1, 1), (E4M3, BF16, 256, 1024, 32, 8, 128, 16, 1, 1),
         (E4M3, F16, 64, 8000, 32, 8, 128, 16, 1, 1), (E4M3, F16, 256, 1024, 32, 8, 128, 64, 1, 1),
         (E4M3, BF16, 256, 1024, 32, 8, 64, 64, 1, 2), (E4M3, F16, 256, 1024, 16, 8, 64, 16, 1, 2),
         (E4M3, BF16, 1, 4096, 32, 32, 128, 16, 1, 1), (E4M3, BF16, 1, 2048, 32, 32, 64, 64, 1, 2),
         (BF16, BF16, 256, 1024, 32, 8, 128, 16, 2, 2), (F16, F16, 512, 512, 32, 8, 64, 16, 2, 2),
         (BF16, BF16, 512, 512, 32, 8, 64, 16, 2, 2), (BF16, BF16, 1, 2048, 32, 32, 128, 16, 2, 2)]


def check(kv, act, B, L, Hq, Hkv, D, ps, weights, diff):
    plain, w, d = plans(kv, act, B, L, Hq, Hkv, D, ps)
    assert (plain.ctas_per_sm, w.ctas_per_sm, d.ctas_per_sm) == (2, weights, diff)
    assert w.capacity_tokens >= L and d.capacity_tokens >= L
    if weights == 2:
        assert w.as_dict() == plain.as_dict()


@pytest.mark.parametrize("case", CASES)
def test_two_ctas_only_where_they_are_resident(fdlib, case):
    check(*case)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_the_device_says_the_same(fdlib, case):
    check(*case)


@pytest.mark.parametrize("kv", [E4M3, BF16])
@pytest.mark.parametrize("opts", [dict(), dict(max_seq_len=1500), dict(num_splits=3),
                                  dict(ctas_per_sm=2, tile_tokens=64), dict(q_len=3)])
def test_decoders_plans_cover_the_same_lengths(fdlib, kv, opts):
    if opts.get("q_len") and kv == E4M3:
        opts = dict(opts, max_seq_len=1300)
    p = _lib.make_problem(256, 32, 8, 128, 16, 100, 25600, BF16, kv)
    dec = fd.PagedDecoder(p, [1024] * 256, device="cpu", num_sms=152, track_weights=True, **opts)
    want = min(dec.plan.capacity_tokens, 1600)
    assert dec.weights_plan.capacity_tokens >= want
    own = dec.weights_plan.as_dict() != dec.plan.as_dict()
    assert own == (kv == E4M3 and opts in (dict(), dict(max_seq_len=1500), dict(num_splits=3)))
    assert (dec.weights_state is dec.workspace) == (not own)
    assert dec.weights_state.nbytes >= dec.weights_plan.workspace_bytes
    assert dec.weights_workspace.nbytes >= _lib.fd_decode_weights_workspace(dec.weights_plan)


def test_refusals(fdlib):
    p = _lib.make_problem(2, 8, 2, 128, 16, 8, 64, BF16, BF16)
    with pytest.raises(_lib.FdError) as e:
        _lib.fd_plan_weights(p, [10], num_sms=152, shared_kv=1)
    assert e.value.code == _lib.FD_ERR_UNSUPPORTED
    assert fdlib.fd_plan_weights(None, None, None, None) == _lib.FD_ERR_INVALID_ARG
    with pytest.raises(_lib.FdError) as e:
        _lib.fd_plan_weights(p, [10, -1], num_sms=152)
    assert e.value.code == _lib.FD_ERR_INVALID_ARG

"""bf16 parts of a softmax weight over bf16 pools: two (16 bits) behind shared
prefixes, as in the decode of whole sequences, unless one is asked for; one in
cross attention of many query rows unless two are.

V is +1 and -1 in turn and the scores are small, so that outputs nearly cancel
and a weight rounded to 8 bits shows."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.cache_ref import seq_tokens, values
from tests.shared_ref import Cross, Prefix, attend_many, check
from tests.test_gpu_shared_weights import PAIRS, alternate, within_pairs

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D,T", [(64, 20), (64, 90), (128, 20), (128, 90)])
def test_cross(fdlib, D, T, splits):
    """One row tile and two, whole rows and chunks, ends inside tiles."""
    c = Cross(41, [2, 16, 130, 300, 0, 601], T=T, Hq=4, Hkv=2, D=D, kv=BF16, q_mult=0.1)
    alternate(c)
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, num_splits=splits,
                                    weight_parts=2)
    assert dec.plan.weight_parts == 2 and not dec.plan.has_few
    out, lse = dec(**d)
    dec.check()
    within_pairs(c, out.cpu(), lse.cpu(), "two parts")
    one = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, num_splits=splits)
    assert one.plan.weight_parts == 1
    out1, lse1 = one(**d)
    one.check()
    c.verify(out1, lse1, what="one part")
    assert torch.equal(lse1, lse)  # the denominators' weights are not rounded


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D,T", [(64, 1), (128, 1), (128, 3)])
def test_prefixes(fdlib, D, T, splits):
    lens = [T + i % 5 for i in range(40)]
    p = Prefix(42, [2, 16, 130, 601], [i % 5 - 1 for i in range(40)], lens, T=T, Hq=16, Hkv=2, D=D, kv=BF16, q_mult=0.1)
    alternate(p)
    d = p.device()
    make = lambda **kw: fd.PrefixDecoder.for_pools(  # noqa: E731
        d["q"], d["k_pages"], d["v_pages"], d["prefix_table"], p.plens, p.of, d["block_table"], p.lens, num_splits=splits, **kw)
    dec = make()
    assert dec.plan.shared.weight_parts == 2
    out, lse = (x.cpu() for x in dec(**d))
    dec.check()
    out, lse = out.view(p.q.shape), lse.view(p.q.shape[:-1])
    k, v = values(p.k, p.ks), values(p.v, p.vs)
    for b, L in enumerate(p.lens):
        kk, vv = seq_tokens(k, p.table[b], L, p.ps), seq_tokens(v, p.table[b], L, p.ps)
        if p.of[b] >= 0:
            g = p.of[b]
            kk = torch.cat([seq_tokens(k, p.ptable[g], p.plens[g], p.ps), kk])
            vv = torch.cat([seq_tokens(v, p.ptable[g], p.plens[g], p.ps), vv])
        ref = attend_many(p.q[b].double(), kk, vv, [kk.shape[0] - T + 1 + t for t in range(T)])
        check(out[b], lse[b], ref, kk.shape[0], PAIRS, BF16, what=f"sequence {b}")
    one = make(weight_parts=1)
    out, lse = one(**d)
    one.check()
    p.verify(out, lse, what="one part")


def test_large_and_hidden_values(fdlib):
    """Scores of some hundreds, and infinities behind the last token."""
    c = Cross(43, [1000, 260, 17], T=70, Hq=4, Hkv=2, D=128, kv=BF16, q_mult=40.0)
    c.v[torch.isnan(c.v)] = float("inf")
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, weight_parts=2)
    out, lse = dec(**d)
    dec.check()
    c.verify(out, lse, what="large scores")

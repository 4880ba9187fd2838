"""Rounding of the softmax weights where cross attention and the own tokens of
prefixed sequences run on the decode kernel (16-bit pools): hi + lo pairs, 16
bits or more.

V is +1 and -1 alternately and the scores are small, so that outputs nearly
cancel: a weight rounded to 11 bits alone shows."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.cache_ref import seq_tokens, values
from tests.shared_ref import Cross, Prefix, attend_many, check

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
KINDS = [F16, BF16]
IDS = ["f16", "bf16"]
PAIRS = 2.0 ** -16  # r_p of weights as pairs (bf16 2^-17, f16 2^-22 and less)


def alternate(c):
    """V of every live token +1 or -1 in turn (E4M3: times its page's scale)."""
    live = ~torch.isnan(values(c.v, c.vs))
    sign = 1.0 - 2.0 * (torch.arange(c.ps) % 2)
    c.v[live] = sign[None, :, None, None].expand(c.v.shape)[live].to(c.v.dtype)


def few(c):
    """The case through the decode kernel."""
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, beams=c.beams)
    assert dec.plan.has_few
    out, lse = dec(**d)
    dec.check()
    return out.cpu(), lse.cpu()


def within_pairs(c, out, lse, what):
    k, v = values(c.k, c.ks), values(c.v, c.vs)
    for r, L in enumerate(c.kv_lens):
        kk, vv = seq_tokens(k, c.table[r], L, c.ps), seq_tokens(v, c.table[r], L, c.ps)
        check(out[r], lse[r], attend_many(c.q[r].double(), kk, vv), L, PAIRS, c.q_dtype, what=f"{what} row {r}")


@pytest.mark.parametrize("kv", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 4])
def test_few_rows(fdlib, kv, D, T):
    c = Cross(31, [2, 4, 6, 10, 16, 30, 2, 4, 40, 8], T=T, Hq=8, Hkv=2, D=D, kv=kv, q_mult=0.15)
    alternate(c)
    out, lse = few(c)
    within_pairs(c, out, lse, "few rows")


@pytest.mark.parametrize("kv", KINDS, ids=IDS)
@pytest.mark.parametrize("T", [1, 4])
def test_own_tokens(fdlib, kv, T):
    """Sequences behind no prefix: the own pass alone."""
    p = Prefix(32, [16], [-1] * 8, [4, 6, 8, 10, 16, 30, 40, 4], T=T, Hq=8, Hkv=2, D=64, kv=kv, q_mult=0.15)
    alternate(p)
    d = p.device()
    dec = fd.PrefixDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["prefix_table"], p.plens, p.of,
                                     d["block_table"], p.lens)
    out, lse = dec(**d)
    dec.check()
    out, lse = out.cpu().view(p.q.shape), lse.cpu().view(p.q.shape[:-1])
    k, v = values(p.k, p.ks), values(p.v, p.vs)
    for b, L in enumerate(p.lens):
        kk, vv = seq_tokens(k, p.table[b], L, p.ps), seq_tokens(v, p.table[b], L, p.ps)
        ref = attend_many(p.q[b].double(), kk, vv, [L - T + 1 + t for t in range(T)])
        check(out[b], lse[b], ref, L, PAIRS, p.q_dtype, what=f"own tokens of {b}")

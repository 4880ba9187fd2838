"""Limits of device-side waits (timeout_us) of cross attention and shared
prefixes: a limit that ends a wait for something that does not come leaves a
call alone whose parts only take longer than that."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.shared_ref import Cross, Prefix

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_items_longer_than_the_limit(fdlib, kv):
    """One chunk of 40000 tokens (313 tiles of at least 1.3 us) under a limit
    of 100 us: the next item's query rows are waited for all the while."""
    c = Cross(21, [40000, 300], T=140, Hq=1, Hkv=1, D=64, kv=kv, ps=128)
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, num_splits=1,
                                    timeout_us=100)
    assert dec.plan.num_splits == 1
    for _ in range(3):
        out, lse = dec(**d)
        dec.check()
    c.verify(out, lse, what="long items")


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_own_tokens_longer_than_the_limit(fdlib, kv):
    """The own tokens' pass ends 0.7 ms late on 122 SMs (by its consumers, which
    none of its own waits meets) under a limit of 100 us: meanwhile the
    pass over the prefixes has other SMs, and more items than CTAs."""
    n = 60
    p = Prefix(22, [20 + i % 90 for i in range(n)] + [8192], list(range(n + 1)), [1 + i % 9 for i in range(n + 1)], Hq=4,
               Hkv=2, D=64, kv=kv)
    d = p.device()
    dec = fd.PrefixDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["prefix_table"], p.plens, p.of, d["block_table"],
                                     p.lens, num_splits=64, timeout_us=100, debug_stall_us=700, debug_stall_role=2)
    assert dec.plan.own.grid_ctas == 2 * (n + 1) and dec.plan.shared.num_splits == 64
    assert dec.plan.shared.timeout_us == 100 and dec.plan.shared.debug_stall_us == 0
    for _ in range(3):
        out, lse = dec(**d)
        dec.check()
    p.verify(out, lse, what="late own tokens")

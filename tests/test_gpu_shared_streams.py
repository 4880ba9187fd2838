"""A decoder made on a busy stream and called on another one at once: its
workspace is filled with zeros before the call."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.shared_ref import Cross, Prefix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40])
def test_made_on_a_busy_stream(fdlib, T):
    c = Cross(51, [300, 700], T=T, Hq=4, Hkv=2, D=64)
    p = Prefix(52, [300, 40], [0, 1, 0, -1], [9, 20, 3, 40], Hq=4, Hkv=2, D=64)
    cd, pd = c.device(), p.device()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dirty = [torch.full((1 << 22,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    del dirty
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    cross = fd.CrossDecoder.for_pools(cd["q"], cd["k_pages"], cd["v_pages"], cd["block_table"], c.kv_lens, num_splits=2)
    with torch.cuda.stream(side):
        out, lse = cross(**cd)
    torch.cuda._sleep(20_000_000)
    prefix = fd.PrefixDecoder.for_pools(pd["q"], pd["k_pages"], pd["v_pages"], pd["prefix_table"], p.plens, p.of,
                                        pd["block_table"], p.lens, num_splits=2)
    with torch.cuda.stream(side):
        pout, plse = prefix(**pd)
    cross.check()
    prefix.check()
    c.verify(out, lse, what="cross")
    p.verify(pout, plse, what="prefix")

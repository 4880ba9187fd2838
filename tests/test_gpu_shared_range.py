"""Cross attention over E4M3 pools where a query row and K's scales are both so
small that their product underflows: the scores are 0, not NaN."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.shared_ref import Cross

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("mult,scale", [(1e-34, 1e-8), (1e-30, 1e-15), (1e-38, 1e-30), (1e-37, 1e8)])
def test_tiny_queries_and_scales(fdlib, T, mult, scale):
    """The last tiles are partial, and one row's pages mix tiny scales with
    ordinary ones."""
    c = Cross(23, [200, 77, 130], T=T, Hq=4, Hkv=2, D=64, kv=E4M3, ps=16)
    c.q = (c.q.float() * mult).to(BF16)
    c.ks[c.table[:2][c.table[:2] >= 0].long()] *= scale
    c.ks[c.table[2][:4].long()] *= scale
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens)
    out, lse = dec(**d)
    dec.check()
    c.verify(out, lse, what=f"queries * {mult}, scales * {scale}")

"""Cross attention over E4M3 pools whose V scales differ by much within a chunk:
the weights are pairs of bf16 there, 16 bits, under bf16 queries too.

V is +1 and -1 in turn times its page's scale and the scores are small, so that
outputs nearly cancel and a weight rounded to 8 bits shows."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.shared_ref import Cross
from tests.test_gpu_shared_weights import alternate, within_pairs

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("q", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_very_different_sizes(fdlib, q, D):
    """Prompts over E4M3 pages whose V scales differ by 2^6 within a chunk."""
    c = Cross(33, [32, 48, 96, 300], T=40, Hq=4, Hkv=2, D=D, kv=E4M3, q=q, q_mult=0.05)
    alternate(c)
    for r, L in enumerate(c.kv_lens):
        for j in range(-(-L // 16)):
            c.vs[int(c.table[r, j])] = 2.0 ** (-6 * (j % 2))
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens)
    out, lse = dec(**d)
    dec.check()
    within_pairs(c, out.cpu(), lse.cpu(), "wide scales")

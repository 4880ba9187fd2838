"""Cross attention of padded batches with very many sequences on an encoder
row, most of them without a token: the ranges of tokens are found in time."""
import random

import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from tests.cache_ref import seq_tokens, values
from tests.shared_ref import Cross, attend_many, check, r_p

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


def verify_rows(c, out, lse, fill):
    """Cross.verify for many sequences: all live tokens of a KV row at once."""
    out, lse = out.cpu(), lse.cpu()
    k, v = values(c.k, c.ks), values(c.v, c.vs)
    live = torch.arange(c.T)[None] < torch.tensor(c.q_lens)[:, None]
    assert bool((out[~live] == fill).all()) and bool((lse[~live] == fill).all())
    for r, L in enumerate(c.kv_lens):
        mine = live.clone()
        mine[:r * c.beams] = False
        mine[(r + 1) * c.beams:] = False
        kk, vv = seq_tokens(k, c.table[r], L, c.ps), seq_tokens(v, c.table[r], L, c.ps)
        if bool(mine.any()):
            check(out[mine], lse[mine], attend_many(c.q[mine].double(), kk, vv), L, r_p(c.q_dtype, c.kv), c.q_dtype,
                  what=f"row {r}", vmax=float(vv.abs().max()) if L and c.kv != BF16 else 0.0)


def run(c, **opts):
    d = c.device()
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens, beams=c.beams, **opts)
    for _ in range(2):
        out, lse = torch.full_like(d["q"], 7.0), torch.full(d["q"].shape[:-1], 7.0, device="cuda")
        dec(**d, out=out, lse=lse)
        dec.check()
    verify_rows(c, out, lse, 7.0)


@pytest.mark.parametrize("kv,q", [(BF16, BF16), (E4M3, F16)], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows,beams,T,heads", [(3, 257, 3, (2, 1)), (2, 1000, 9, (3, 1)), (40, 300, 2, (2, 2)),
                                                (70, 31, 5, (4, 1)), (1, 5000, 1, (1, 1))])
def test_ragged(fdlib, rows, beams, T, heads, kv, q):
    """Long runs of sequences without tokens between single ones and full ones."""
    rng = random.Random(rows)
    counts = []
    while len(counts) < rows * beams:
        kind = rng.choice(["none", "none", "some", "full", "one"])
        n = rng.randint(1, 400)
        counts += [{"none": 0, "some": rng.randint(0, T), "full": T, "one": 1}[kind] for _ in range(n)]
    lens = [rng.choice([0, 1, 40, 130]) if i else 140 for i in range(rows)]
    c = Cross(24, lens, beams=beams, T=T, Hq=heads[0], Hkv=heads[1], D=64, kv=kv, q=q, q_lens=counts[:rows * beams])
    run(c)


def test_within_a_short_limit(fdlib):
    """60000 sequences, 1200 of them with a token, under a limit of 3 ms."""
    beams = 60000
    c = Cross(25, [100], beams=beams, T=1, Hq=1, Hkv=1, D=64, kv=BF16, q_lens=[int(i % 50 == 49) for i in range(beams)])
    run(c, timeout_us=3000)

"""Cross attention (CrossDecoder, fd_cross_paged) against the float64
definition, with NaN behind every length and in every unused page."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests.shared_ref import Cross

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
KINDS = [(F16, F16), (BF16, BF16), (E4M3, BF16), (E4M3, F16)]
IDS = ["f16", "bf16", "e4m3-bf16", "e4m3-f16"]


def run(c, plan_lens=None, want_lse=True, fill=7.0, both=True, **opts):
    d = c.device()
    q_lens = d.pop("q_lens")
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], plan_lens or c.kv_lens,
                                    beams=c.beams, **opts)
    out = torch.full_like(d["q"], fill)
    lse = torch.full(d["q"].shape[:-1], fill, device="cuda") if want_lse else None
    dec(**d, q_lens=q_lens, out=out, lse=lse, want_lse=want_lse)
    dec.check()
    if both and dec.plan.has_few and q_lens is None:
        # the decode kernel took the call; given counts, the other kernel takes it
        out2, lse2 = dec(**d, q_lens=torch.full((len(c.q),), c.T, dtype=torch.int32, device="cuda"))
        dec.check()
        c.verify(out2, lse2, what="the same, with counts")
    return out, lse, dec


@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens(fdlib, kv, q, D):
    """Lengths of zero, one, around pages and tiles; one token each."""
    c = Cross(1, [0, 1, 15, 16, 17, 127, 128, 129, 300, 513], Hq=8, Hkv=2, D=D, kv=kv, q=q, ps=32)
    out, lse, _ = run(c)
    c.verify(out, lse, what="single tokens")


@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T", [(2, 2, 130), (8, 2, 70), (5, 1, 27), (6, 2, 300), (12, 1, 33)])
def test_prompts(fdlib, kv, q, D, Hq, Hkv, T):
    """More query rows than a tile holds, groups that do not divide one."""
    c = Cross(2, [77, 0, 260, 5], T=T, Hq=Hq, Hkv=Hkv, D=D, kv=kv, q=q)
    out, lse, _ = run(c)
    c.verify(out, lse, what="prompts")


@pytest.mark.parametrize("ps", [16, 32, 48, 64, 128, 176, 256])
@pytest.mark.parametrize("kv,q", KINDS[1:3], ids=IDS[1:3])
def test_page_sizes(fdlib, kv, q, ps):
    c = Cross(3, [401, 176, 129], T=9, Hq=4, Hkv=2, D=128, kv=kv, q=q, ps=ps)
    out, lse, _ = run(c)
    c.verify(out, lse, what=f"page size {ps}")


@pytest.mark.parametrize("beams,T", [(1, 6), (3, 1), (5, 40), (70, 2)])
@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
def test_beams_and_padded_queries(fdlib, beams, T, kv, q):
    """Rows past a sequence's query tokens stay as they were; a sequence may
    have none."""
    lens = [200, 33, 0]
    counts = [(3 * i) % (T + 1) for i in range(len(lens) * beams)]
    c = Cross(4, lens, beams=beams, T=T, Hq=4, Hkv=2, D=64, kv=kv, q=q, q_lens=counts)
    out, lse, _ = run(c)
    c.verify(out, lse, untouched=7.0, what="padded")


@pytest.mark.parametrize("splits", [1, 2, 5, 16])
@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
@pytest.mark.parametrize("T", [1, 40])
def test_splits(fdlib, splits, kv, q, T):
    """KV rows cut into chunks and joined; short rows beside them are not."""
    c = Cross(5, [2100, 900, 0, 130, 1], T=T, Hq=8, Hkv=2, D=128, kv=kv, q=q, ps=64)
    out, lse, dec = run(c, num_splits=splits)
    c.verify(out, lse, what=f"{splits} splits")


def test_lengths_change_within_the_capacity(fdlib):
    c = Cross(6, [50, 700, 300], T=3, Hq=4, Hkv=2, D=64, pad_cols=30)
    out, lse, dec = run(c, plan_lens=[10, 20, 30], max_kv_len=1024)
    c.verify(out, lse, what="grown lengths")


def test_strided_queries_and_no_lse(fdlib):
    c = Cross(7, [99, 200], T=5, Hq=4, Hkv=2, D=64)
    d = c.device()
    wide = torch.randn(2, 5, 3 * 4 * 64, device="cuda").to(torch.bfloat16)
    q = wide[..., 256:512].unflatten(-1, (4, 64))
    q.copy_(d["q"])
    dec = fd.CrossDecoder.for_pools(q, d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens)
    out, lse = dec(q, d["k_pages"], d["v_pages"], d["block_table"], d["kv_lens"], want_lse=False)
    dec.check()
    assert lse is None
    c.verify(out, None, what="strided")


@pytest.mark.parametrize("q", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("D,T", [(64, 40), (128, 3), (128, 90)])
def test_scales_of_very_different_sizes(fdlib, q, D, T):
    """E4M3 pages whose scales differ by up to 2^12, some rows all alike."""
    c = Cross(11, [700, 16, 129, 1], T=T, Hq=6, Hkv=2, D=D, kv=E4M3, q=q, ps=32, wide=True, q_mult=0.1)
    for splits in (1, 3):
        out, lse, _ = run(c, num_splits=splits)
        c.verify(out, lse, what="wide scales")


def test_scales_that_are_not_positive(fdlib):
    """A page of negative scales and one of zeros."""
    c = Cross(12, [300, 90], T=70, Hq=4, Hkv=2, D=64, kv=E4M3, ps=32)
    c.ks[int(c.table[0, 2])] *= -1
    c.vs[int(c.table[0, 3])] *= -1
    c.ks[int(c.table[1, 2])] = 0  # the page the second row ends in
    c.vs[int(c.table[0, 5])] = 0
    c.wide = True
    out, lse, _ = run(c)
    c.verify(out, lse, what="scales")


@pytest.mark.parametrize("mult", [1e-30, 1e-6, 3e4, 1e20])
def test_query_range_over_e4m3(fdlib, mult):
    """bf16 queries far from f16's range over E4M3 keys of the opposite size."""
    c = Cross(13, [200, 77], T=70, Hq=4, Hkv=2, D=64, kv=E4M3, ps=16)
    c.q = (c.q.float() * mult).to(BF16)
    c.ks /= mult
    out, lse, _ = run(c)
    c.verify(out, lse, what="query range")


@pytest.mark.parametrize("T", [3, 30])
def test_nan_codes_stay_in_their_head(fdlib, T):
    """A live NaN code reaches every row of its KV head and none of the others."""
    c = Cross(14, [200, 77], T=T, Hq=4, Hkv=2, D=64, kv=E4M3, ps=16)
    ref, _, _ = run(c)
    c.v.view(torch.uint8)[int(c.table[0, 1]), 3, 1, 5] = 0x7f
    c.k.view(torch.uint8)[int(c.table[1, 0]), 2, 0, 9] = 0xff
    out, lse, _ = run(c, both=False)
    assert bool(torch.isnan(out[0, :, 2:, 5]).all()) and bool(torch.isnan(out[1, :, :2]).all())
    out[0, :, 2:, 5], ref[0, :, 2:, 5] = 0, 0
    out[1, :, :2], ref[1, :, :2] = 0, 0
    assert torch.equal(out, ref)


def test_large_scores(fdlib):
    """Scores of some hundreds: the running maximum moves, nothing overflows."""
    for kv in (F16, BF16):
        c = Cross(8, [1000, 260], T=70, Hq=4, Hkv=2, D=128, kv=kv, q_mult=40.0)
        out, lse, _ = run(c)
        c.verify(out, lse, what="large scores")


def test_rising_maximum(fdlib):
    """Keys that grow along the row: every tile passes the reference maximum."""
    c = Cross(9, [900], T=40, Hq=4, Hkv=2, D=64)
    ramp = torch.linspace(0.1, 12.0, 900)
    for j in range(57):
        page = int(c.table[0, j])
        n = min(16, 900 - 16 * j)
        c.k[page, :n] = (c.k[page, :n].float() * ramp[16 * j:16 * j + n, None, None]).to(BF16)
    out, lse, _ = run(c)
    c.verify(out, lse, what="rising maximum")


@pytest.mark.parametrize("T", [4, 40])
def test_device_errors_are_reported(fdlib, T):
    """Lengths beyond the capacity, pages and query counts out of range: the
    status says so, the other sequences are right, nothing else is touched."""
    c = Cross(10, [100, 60, 90], T=T, Hq=4, Hkv=2, D=64)
    d = c.device()
    ql = d.pop("q_lens")
    assert ql is None
    dec = fd.CrossDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["block_table"], c.kv_lens)

    def call(bit, good, **kw):
        out = torch.full_like(d["q"], 7.0)
        dec(**{**d, **kw}, out=out)
        assert int(dec.status.item()) & bit  # a cut length may meet unused pages: their bit as well
        with pytest.raises(fd.FdError):
            dec.check()
        ref, _ = dec(**d, q_lens=torch.full_like(d["kv_lens"], T) if "q_lens" in kw else None)
        dec.check()
        for b in good:
            assert torch.equal(out[b], ref[b])
        return out

    long = d["kv_lens"].clone()
    long[1] = 5000
    call(_lib.FD_DEV_CAPACITY, [0, 2], kv_lens=long)
    long[1] = -3
    out = call(_lib.FD_DEV_CAPACITY, [0, 2], kv_lens=long)
    assert bool((out[1] == 0).all())
    table = d["block_table"].clone()
    table[2, 1] = 1 << 20
    call(_lib.FD_DEV_BAD_PAGE, [0, 1], block_table=table)
    counts = torch.tensor([T, T + 5, -1], dtype=torch.int32, device="cuda")
    out = call(_lib.FD_DEV_CAPACITY, [0], q_lens=counts)
    assert bool((out[1:] == 7.0).all())

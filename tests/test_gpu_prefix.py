"""Decode behind shared prefixes (PrefixDecoder, fd_decode_paged_prefix)
against the float64 definition, with NaN behind every length and in every
unused page."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests.shared_ref import Prefix

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
KINDS = [(F16, F16), (BF16, BF16), (E4M3, BF16), (E4M3, F16)]
IDS = ["f16", "bf16", "e4m3-bf16", "e4m3-f16"]


def decoder(c, d, **opts):
    return fd.PrefixDecoder.for_pools(d["q"], d["k_pages"], d["v_pages"], d["prefix_table"], c.plens, c.of,
                                      d["block_table"], c.lens, **opts)


def run(c, **opts):
    d = c.device()
    dec = decoder(c, d, **opts)
    out, lse = dec(**d)
    dec.check()
    return out, lse, dec


@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 3])
def test_groups(fdlib, kv, q, D, T):
    """Groups of several sizes in any order, sequences behind no prefix, an
    empty group, prefixes that end inside a page and one of length zero."""
    of = [2, 0, -1, 1, 0, 2, 0, 4, -1, 0, 2, 4]
    lens = [T + (7 * i) % 60 for i in range(len(of))]
    c = Prefix(1, [131, 40, 300, 77, 0], of, lens, T=T, Hq=8, Hkv=2, D=D, kv=kv, q=q)
    out, lse, _ = run(c)
    c.verify(out, lse, what="groups")


@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
def test_more_rows_than_a_tile(fdlib, kv, q):
    c = Prefix(2, [500], [0] * 90, [1 + i % 40 for i in range(90)], Hq=10, Hkv=2, D=64, kv=kv, q=q, ps=32)
    out, lse, _ = run(c)
    c.verify(out, lse, what="many rows")


@pytest.mark.parametrize("splits", [1, 3, 9])
@pytest.mark.parametrize("kv,q", KINDS, ids=IDS)
def test_splits(fdlib, splits, kv, q):
    c = Prefix(3, [1500, 200], [0, 1, 0, 0, -1, 1], [5, 9, 300, 1, 20, 64], Hq=4, Hkv=1, D=128, kv=kv, q=q, ps=64)
    out, lse, _ = run(c, num_splits=splits)
    c.verify(out, lse, what=f"{splits} splits")


def test_sequences_without_own_tokens(fdlib):
    """Own lengths of zero: the prefix alone; without a prefix either, zeros."""
    c = Prefix(4, [90], [0, -1, 0], [0, 0, 12], Hq=4, Hkv=2, D=64)
    out, lse, _ = run(c)
    c.verify(out, lse, what="no own tokens")
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())


def test_regroup(fdlib):
    c = Prefix(5, [90, 200, 33], [0, 1, 2, 0, 1], [4, 5, 6, 7, 8], Hq=4, Hkv=2, D=64)
    d = c.device()
    dec = decoder(c, d)
    for of in ([2, 2, -1, 0, 0], [-1] * 5, [1] * 5):
        c.of = of
        dec.regroup(of)
        out, lse = dec(**d)
        dec.check()
        c.verify(out, lse, what=str(of))


def test_bad_groups_are_reported(fdlib):
    c = Prefix(6, [90, 50], [0, 1, 0, 1], [4, 5, 6, 7], Hq=4, Hkv=2, D=64)
    d = c.device()
    dec = decoder(c, d)
    ref, _ = dec(**d)
    dec.check()
    members, offsets = dec.members.clone(), dec.offsets.clone()
    dec.members[1] = 99  # sequence 2's place
    out = torch.full_like(d["q"], 7.0)
    dec(**d, out=out)
    with pytest.raises(fd.FdError) as e:
        dec.check()
    assert e.value.code == _lib.FD_ERR_BAD_PAGE
    assert bool((out[2] == 7.0).all()) and torch.equal(out[[0, 1, 3]], ref[[0, 1, 3]])
    dec.members.copy_(members)
    for bad in ([0, 9, 4], [0, 3, 2], [0, -5, 4], [1, 2, 4]):
        dec.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        dec(**d)
        with pytest.raises(fd.FdError) as e:
            dec.check()
        assert e.value.code == _lib.FD_ERR_BAD_PAGE, bad
    dec.offsets.copy_(offsets)
    out, _ = dec(**d)
    dec.check()
    assert torch.equal(out, ref)

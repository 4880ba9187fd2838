"""Numbers that do not fit the C interface's ints are refused, not cut to 32
bits (2^32 first tokens to keep would be none), and so are fractions."""
import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests.test_cache_op_args import B, D, HKV, MB, NP, PS, append_kw, prob, z


def evict_kw(**kw):
    a = dict(k_pages=z(NP, PS, HKV, D), v_pages=z(NP, PS, HKV, D), block_table=z(B, MB, dtype=torch.int32),
             seq_lens=z(B, dtype=torch.int32), weights=z(B, HKV, 50, dtype=torch.float32), budget=20)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,msg", [
    (dict(sinks=1 << 32), "sinks must"), (dict(sinks=(1 << 32) + 4), "sinks must"), (dict(recent=1 << 33), "recent must"),
    (dict(recent=-(1 << 32)), "recent must"), (dict(sinks=1.5), "sinks must"), (dict(recent=float("inf")), "."),
    (dict(budget=20.5), "budget must"), (dict(budget=(1 << 32) + 20), "budget 4294967316 of a table for 64"),
    (dict(budget=PS * MB + 1), "budget 65 of"), (dict(budget=-1), "budget must"),
    (dict(weights=torch.empty(B, HKV, (1 << 32) + 50, device="meta")), "last dimension of weights must"),
])
def test_evict(fdlib, kw, msg):
    with pytest.raises((ValueError, OverflowError, _lib.FdError), match=msg):
        fd.evict_kv(**evict_kw(**kw))


def test_whole_floats_are_taken(fdlib):
    """A budget computed as a fraction of a length, say: refused only for the host tensors."""
    with pytest.raises(ValueError, match="CUDA"):
        fd.evict_kv(**evict_kw(budget=PS * MB * 0.5, sinks=2.0))


def test_append(fdlib):
    big = torch.empty((1 << 32) + 9, D // 2, device="meta")
    with pytest.raises(ValueError, match="rows of rotary_cos must"):
        fd.append_kv_norm(**append_kw(rotary_cos=big, rotary_sin=big))


def test_decode_weights(fdlib):
    p = prob(max_blocks_per_seq=MB, num_pages=NP)
    dec = fd.PagedDecoder(p, [40, 50], device="cpu", num_sms=152, track_weights=True)
    args = (z(B, 8, D), z(NP, PS, HKV, D), z(NP, PS, HKV, D), z(B, MB, dtype=torch.int32), z(B, dtype=torch.int32))
    with pytest.raises(ValueError, match="last dimension of weights_out must"):
        dec.decode_weights(*args, torch.empty(B, HKV, (1 << 32) + 64, device="meta"))

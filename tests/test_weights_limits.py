"""The largest number of query rows a KV head may have with attention totals."""
import pytest
import torch

from split_kv_decode_paged_gb300 import _lib

BF = torch.bfloat16


def workspace(rows, q_len=1, Hkv=1, lens=(40, 3)):
    p = _lib.make_problem(len(lens), rows * Hkv, Hkv, 64, 16, 4, 16, BF, BF)
    return _lib.fd_decode_weights_workspace(_lib.fd_plan_weights(p, list(lens), num_sms=152, q_len=q_len))


@pytest.mark.parametrize("rows,q_len", [(1, 1), (17, 1), (6141, 1), (6142, 1), (6144, 1), (96, 64), (2048, 3)])
def test_up_to_6144_query_rows(fdlib, rows, q_len):
    n = rows * q_len
    assert workspace(rows, q_len) >= 2 * n * 4 * (1 + 40)


@pytest.mark.parametrize("rows,q_len", [(6145, 1), (6148, 1), (97, 64), (1 << 19, 64)])
def test_no_more_than_6144_query_rows(fdlib, rows, q_len):
    with pytest.raises(_lib.FdError) as e:
        workspace(rows, q_len)
    assert e.value.code == _lib.FD_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [6141, 6144])
def test_totals_of_6144_query_rows(fdlib, rows):
    from tests.test_gpu_weights import check
    check("bf16", "bf16", [40, 3, 0], rows, 1, 64, 16, seed=rows)

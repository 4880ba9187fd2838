"""A call whose launches fail is made once: FdError at once, and not the whole
operator a second time over totals that were already added or rows that moved.
The failure is a stand-in for libfd's entry point that counts its calls and
returns a status; nothing is launched."""
import ctypes

import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests.test_gpu_weights import setup

pytestmark = pytest.mark.gpu


@pytest.fixture
def failing(fdlib):
    """Puts a function that returns `status` in the place of all four entry
    points (of the native way); the second list counts the Python way's calls."""
    fast = _lib.fast()
    assert fast
    names = ("fd_append_kv_norm", "fd_evict_kv", "fd_decode_paged_weights", "fd_decode_paged_diff")
    real = [ctypes.cast(getattr(fdlib, n), ctypes.c_void_p).value for n in names]
    calls, again = [], []
    keep = []

    def put(status, monkeypatch):
        @ctypes.CFUNCTYPE(ctypes.c_int)
        def stub():
            calls.append(status)
            return status
        keep.append(stub)
        fast.init(*[ctypes.cast(stub, ctypes.c_void_p).value] * 4, _lib.FdError)
        for n in names:
            monkeypatch.setattr(_lib, n, lambda *a, **kw: again.append(a))
        return calls, again
    yield put
    fast.init(*real, _lib.FdError)


def all_four():
    lens = [40, 9]
    q, kp, vp, _, _, bt = (None if t is None else t.cuda() for t in setup("bf16", "bf16", lens, 8, 2, 64, 16))
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    w = torch.rand(2, 2, 64).cuda()
    dec = fd.PagedDecoder.for_pools(q, kp, vp, bt, lens, track_weights=True)
    dif = fd.DiffDecoder.for_pools(q, kp, vp, bt, lens)
    new = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    return [lambda: fd.append_kv_norm(q, new, new, kp, vp, bt, dl), lambda: fd.evict_kv(kp, vp, bt, dl, w, 20, weights_out=w),
            lambda: dec.decode_weights(q, kp, vp, bt, dl, w), lambda: dif(q, kp, vp, bt, dl, torch.ones(8).cuda())]


def test_failed_calls_raise_and_are_not_repeated(failing, monkeypatch):
    todo = all_four()
    calls, again = failing(_lib.FD_ERR_CUDA, monkeypatch)
    for i, f in enumerate(todo):
        with pytest.raises(_lib.FdError) as e:
            f()
        assert e.value.code == _lib.FD_ERR_CUDA and "fd_" in str(e.value)
        assert len(calls) == i + 1 and not again


@pytest.mark.parametrize("status", ["FD_ERR_INVALID_ARG", "FD_ERR_UNSUPPORTED", "FD_ERR_WORKSPACE_TOO_SMALL"])
def test_refused_calls_go_the_python_way(failing, monkeypatch, status):
    todo = all_four()
    calls, again = failing(getattr(_lib, status), monkeypatch)
    for f in todo:
        f()
    assert len(calls) == len(again) == 4

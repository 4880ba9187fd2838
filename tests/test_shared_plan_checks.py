"""Cross attention and decode behind shared prefixes: plans whose two parts do
not describe the same pools, or whose chunks overflow, are refused before
anything is launched (no GPU)."""
import pytest

from split_kv_decode_paged_gb300 import _lib
from tests.test_shared_args import INVALID, SMALL, _raw_cross, _raw_prefix, problem

pytestmark = pytest.mark.usefixtures("fdlib")


def _few_plan():
    plan = _lib.fd_plan_cross(problem(), [100, 20], num_sms=152)
    assert plan.has_few
    return plan


@pytest.mark.parametrize("field,value", [("q_dtype", _lib.FD_F16), ("kv_dtype", _lib.FD_F16), ("page_size", 32),
                                         ("num_pages", 1 << 20)])
def test_own_plan_of_other_pools(field, value):
    plan = _lib.fd_plan_prefix(problem(), [5, 9], 8, [30], [0, 2], num_sms=152)
    assert getattr(plan.own.problem, field) != value
    setattr(plan.own.problem, field, value)
    assert _raw_prefix(plan) == INVALID


def test_own_plan_of_more_rows():
    """An own pass that would write more rows than the workspace has."""
    plan = _lib.fd_plan_prefix(problem(), [5, 9], 8, [30], [0, 2], num_sms=152)
    plan.own.row_fold, plan.own.problem.B = 2, 4
    assert _raw_prefix(plan) == INVALID


def test_few_plan_with_causal_tokens():
    plan = _lib.fd_plan_cross(problem(), [100, 20], tokens=3, num_sms=152)
    assert plan.has_few and plan.few.q_len <= 1
    plan.few.q_len = 3
    assert _raw_cross(plan) == INVALID


@pytest.mark.parametrize("make", [lambda: _lib.fd_plan_cross(problem(), [100, 20], tokens=40, num_sms=152),
                                  lambda: _lib.fd_plan_prefix(problem(), [5, 9], 8, [30], [0, 2], num_sms=152)],
                         ids=["cross", "prefix"])
def test_chunks_that_overflow(make):
    plan = make()
    shared = getattr(plan, "shared", plan)
    shared.chunk_tokens = (1 << 31) - 128  # length + chunk leaves 31 bits
    assert (_raw_cross if shared is plan else _raw_prefix)(plan) == INVALID


def test_chunk_of_the_largest_table():
    """A capacity of 2^30 tokens with rows enough that partial states fit only
    for few chunks: the planned chunk is one that the call takes."""
    p = problem(B=64, page_size=1 << 20, max_blocks_per_seq=1 << 10)
    plan = _lib.fd_plan_cross(p, [(1 << 30) * 9 // 10] * 64, tokens=1000, num_splits=1, max_kv_len=1 << 30, num_sms=152)
    assert plan.chunk_tokens * plan.num_splits >= 1 << 30 and plan.chunk_tokens <= 1 << 30
    assert _raw_cross(plan, q=None) == INVALID  # (the pointer)
    assert _raw_cross(plan, nb=0) == SMALL      # the plan itself is taken

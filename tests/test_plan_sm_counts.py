"""SM counts that no device has are refused by every planner; the cost model
keeps a queue entry for each CTA of them (and 2^30 SMs of two CTAs were an
empty queue, which ended the process)."""
import subprocess
import sys

import pytest

CODE = """
import torch
from split_kv_decode_paged_gb300 import _lib
p = _lib.make_problem(2, 8, 2, 128, 16, 512, 1024, torch.bfloat16, torch.bfloat16)
for f in (_lib.fd_plan, _lib.fd_plan_weights, _lib.fd_plan_diff):
    try:
        f(p, [8000, 5000], num_sms={sms}, **{opts})
        print("planned")
    except _lib.FdError as e:
        print("status", e.code)
"""


def outcome(sms, **opts):
    r = subprocess.run([sys.executable, "-c", CODE.format(sms=sms, opts=opts)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    return r.stdout.split("\n")[:-1]


@pytest.mark.parametrize("sms,opts", [(1 << 30, dict(ctas_per_sm=2, tile_tokens=64)), ((1 << 31) - 1, dict()), (65537, dict())])
def test_refused(fdlib, sms, opts):
    assert outcome(sms, **opts) == ["status 1"] * 3


@pytest.mark.parametrize("sms", [1, 2, 152, 65536])
def test_planned(fdlib, sms):
    assert outcome(sms) == ["planned"] * 3

"""Plans of cross attention and of decode behind shared prefixes: the parts of
a weight, and the structures' layout against the header's (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib
from tests.test_shared_args import INVALID, _raw_cross, code, problem

pytestmark = pytest.mark.usefixtures("fdlib")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _prefix(**kw):
    return _lib.fd_plan_prefix(problem(), [5, 9], 8, [30], [0, 2], num_sms=152, **kw)


@pytest.mark.parametrize("given,cross,prefix", [(0, 1, 2), (1, 1, 1), (2, 2, 2)])
def test_weight_parts(given, cross, prefix):
    assert _lib.fd_plan_cross(problem(), [100, 20], num_sms=152, weight_parts=given).weight_parts == cross
    assert _prefix(weight_parts=given).shared.weight_parts == prefix


@pytest.mark.parametrize("given", [-1, 3])
def test_weight_parts_out_of_range(given):
    assert code(_lib.fd_plan_cross, problem(), [100, 20], num_sms=152, weight_parts=given) == INVALID
    assert code(_prefix, weight_parts=given) == INVALID
    plan = _lib.fd_plan_cross(problem(), [100, 20], num_sms=152)
    plan.weight_parts = given
    assert _raw_cross(plan) == INVALID


def test_weight_parts_is_a_whole_number():
    with pytest.raises(ValueError, match="weight_parts"):
        _lib.fd_plan_cross(problem(), [100, 20], num_sms=152, weight_parts=1.5)
    with pytest.raises(ValueError, match="weight_parts"):
        _prefix(weight_parts=1.5)


def test_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"fd_cross_options": _lib.FdCrossOptions, "fd_cross_plan_t": _lib.FdCrossPlan,
               "fd_prefix_plan_t": _lib.FdPrefixPlan}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fd_api.h"', "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        cname, field, at = line.split()
        py = structs[cname]
        assert int(at) == (ctypes.sizeof(py) if field == "size" else getattr(py, field).offset), (cname, field)


def test_empty_batches():
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16)
    pages = torch.zeros(64, 16, 2, 128, dtype=torch.bfloat16)
    table, ptable = torch.zeros(0, 8, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.int32)
    for lens in ([], torch.zeros(0, dtype=torch.int32)):
        for make in (lambda: fd.CrossDecoder.for_pools(q, pages, pages, table, lens, num_sms=152),
                     lambda: fd.PrefixDecoder.for_pools(q, pages, pages, ptable, [30], lens, table, lens, num_sms=152)):
            with pytest.raises(fd.FdError) as e:
                make()
            assert e.value.code == INVALID

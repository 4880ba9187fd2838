"""Cross attention and decode behind shared prefixes: what the planners, the
C entry points and the binding refuse before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

import split_kv_decode_paged_gb300 as fd
from split_kv_decode_paged_gb300 import _lib

pytestmark = pytest.mark.usefixtures("fdlib")

INVALID, UNSUPPORTED, SMALL = _lib.FD_ERR_INVALID_ARG, _lib.FD_ERR_UNSUPPORTED, _lib.FD_ERR_WORKSPACE_TOO_SMALL


def problem(**kw):
    base = dict(B=2, Hq=8, Hkv=2, D=128, page_size=16, max_blocks_per_seq=8, num_pages=64, q_dtype=torch.bfloat16,
                kv_dtype=torch.bfloat16)
    base.update(kw)
    return _lib.make_problem(**base)


def code(fn, *a, **kw):
    with pytest.raises(fd.FdError) as e:
        fn(*a, **kw)
    return e.value.code


@pytest.mark.parametrize("kw,opts,want", [
    (dict(page_size=24), {}, INVALID),
    (dict(Hq=6, Hkv=4), {}, INVALID),
    (dict(D=96), {}, UNSUPPORTED),
    (dict(q_dtype=torch.float16), {}, UNSUPPORTED),
    (dict(out_dtype=torch.float32), {}, UNSUPPORTED),
    ({}, dict(tokens=-1), INVALID),
    ({}, dict(beams=-2), INVALID),
    ({}, dict(beams=1 << 17), UNSUPPORTED),
    ({}, dict(tokens=1 << 22), UNSUPPORTED),
    (dict(Hq=1 << 16, Hkv=1 << 16), dict(tokens=4096), UNSUPPORTED),
    ({}, dict(num_splits=-1), INVALID),
    ({}, dict(num_sms=(1 << 16) + 1), INVALID),
    ({}, dict(timeout_us=-1), INVALID),
    ({}, dict(debug_stall_us=1000001), INVALID),
    ({}, dict(max_kv_len=129), INVALID),
])
def test_plan_cross_refuses(kw, opts, want):
    assert code(_lib.fd_plan_cross, problem(**kw), [100, 20], **{"num_sms": 152, **opts}) == want


def test_plan_cross_lengths():
    assert code(_lib.fd_plan_cross, problem(), [100, -1], num_sms=152) == INVALID
    assert code(_lib.fd_plan_cross, problem(), [100, 129], num_sms=152) == INVALID
    for bad in ([100], [100, 20, 3], [1.5, 2.0], [[1, 2]], [1, 1 << 31]):
        with pytest.raises(ValueError):
            _lib.fd_plan_cross(problem(), bad, num_sms=152)
    with pytest.raises(ValueError):
        _lib.fd_plan_cross(problem(), [1, 2], num_sms=152, tokens=1 << 33)
    plan = _lib.fd_plan_cross(problem(), [100, 0], tokens=3, beams=5, num_sms=152, max_kv_len=128)
    assert (plan.kv_rows, plan.seqs, plan.tokens, plan.beams) == (2, 10, 3, 5)
    assert plan.capacity_tokens == 128


@pytest.mark.parametrize("kw,opts,want", [
    (dict(page_size=8), {}, INVALID),
    (dict(out_dtype=torch.float32), {}, UNSUPPORTED),
    ({}, dict(shared_kv=1), UNSUPPORTED),
    ({}, dict(q_len=65), INVALID),
    ({}, dict(num_splits=-1), INVALID),
    ({}, dict(max_prefix_len=161), INVALID),
    ({}, dict(prefix_stall_us=-1), INVALID),
    ({}, dict(offsets=[1, 2, 2]), INVALID),
    ({}, dict(offsets=[0, 2, 1]), INVALID),
    ({}, dict(offsets=[0, 2, 3]), INVALID),
    ({}, dict(plens=[30, 161]), INVALID),
    ({}, dict(plens=[30, -1]), INVALID),
    ({}, dict(lens=[5, 129]), INVALID),
    ({}, dict(blocks=0), INVALID),
    ({}, dict(plens=[1] * 8193, offsets=[0] * 8194), UNSUPPORTED),
])
def test_plan_prefix_refuses(kw, opts, want):
    a = dict(lens=[5, 9], blocks=10, plens=[30, 40], offsets=[0, 1, 2])
    a.update({k: opts[k] for k in opts if k in a})
    rest = {k: v for k, v in opts.items() if k not in a}
    got = code(_lib.fd_plan_prefix, problem(**kw), a["lens"], a["blocks"], a["plens"], a["offsets"], num_sms=152, **rest)
    assert got == want


def test_plan_prefix_layout():
    plan = _lib.fd_plan_prefix(problem(), [5, 9], 10, [30, 160], [0, 1, 2], num_sms=152, q_len=3, max_seq_len=100)
    rows = 2 * 3 * 8
    assert plan.ws_own_lse - plan.ws_own_out >= rows * 128 * 4
    assert plan.ws_own - plan.ws_own_lse >= rows * 4
    assert plan.ws_shared - plan.ws_own >= plan.own.workspace_bytes
    assert plan.workspace_bytes - plan.ws_shared >= plan.shared.workspace_bytes
    assert plan.own.capacity_tokens >= 100 and plan.shared.capacity_tokens == 160
    with pytest.raises(TypeError):
        _lib.fd_plan_prefix(problem(), [5, 9], 10, [30, 160], [0, 1, 2], num_sms=152, beams=2)


def _raw_cross(plan, **kw):
    """fd_cross_paged with stand-in pointers: whatever is refused is refused before a launch."""
    at = 1 << 20
    a = dict(q=at, q_stride=8 * 128, q_lens=None, k=at, v=at, ks=None, vs=None, bt=at, kl=at, out=at, lse=at, ws=at,
             nb=1 << 30, st=None)
    a.update(kw)
    return _lib.load().fd_cross_paged(ctypes.byref(plan), a["q"], a["q_stride"], a["q_lens"], a["k"], a["v"], a["ks"],
                                      a["vs"], a["bt"], a["kl"], a["out"], a["lse"], a["ws"], a["nb"], a["st"], None)


def test_cross_call_refuses():
    plan = _lib.fd_plan_cross(problem(), [100, 20], num_sms=152)
    at = 1 << 20
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(kl=None), dict(out=None), dict(ws=None),
               dict(q=at + 8), dict(k=at + 8), dict(out=at + 4), dict(lse=at + 2), dict(ws=at + 128), dict(q_lens=at + 1),
               dict(st=at + 2), dict(ks=at), dict(vs=at), dict(q_stride=1023), dict(q_stride=1028), dict(q_stride=-1024)):
        assert _raw_cross(plan, **kw) == INVALID, kw
    assert _raw_cross(plan, nb=int(plan.workspace_bytes) - 1) == SMALL
    e4m3 = _lib.fd_plan_cross(problem(kv_dtype=torch.float8_e4m3fn), [100, 20], num_sms=152)
    assert _raw_cross(e4m3) == INVALID and _raw_cross(e4m3, ks=at) == INVALID
    for field, value in (("kv_rows", 3), ("seqs", 1 << 23), ("tokens", 0), ("beams", 0), ("num_splits", 0),
                         ("capacity_tokens", 0), ("capacity_tokens", 129), ("timeout_us", -1), ("debug_stall_us", 2000000)):
        bad = _lib.fd_plan_cross(problem(), [100, 20], num_sms=152)
        setattr(bad, field, value)
        assert _raw_cross(bad) == INVALID, field
    other = _lib.fd_plan_prefix(problem(), [5, 9], 8, [30], [0, 2], num_sms=152)
    assert _raw_cross(other.shared) == INVALID


def _raw_prefix(plan, **kw):
    at = 1 << 20
    names = ("q", "k", "v", "ks", "vs", "pt", "pl", "mb", "of", "bt", "sl", "out", "lse", "ws")
    a = {n: at for n in names}
    a.update(ks=None, vs=None, nb=1 << 30)
    a.update(kw)
    return _lib.load().fd_decode_paged_prefix(ctypes.byref(plan), *(a[n] for n in names), a["nb"], a.get("st"), None)


def test_prefix_call_refuses():
    make = lambda: _lib.fd_plan_prefix(problem(), [5, 9], 8, [30], [0, 2], num_sms=152)  # noqa: E731
    at = 1 << 20
    for kw in (dict(q=None), dict(k=None), dict(pt=None), dict(pl=None), dict(mb=None), dict(of=None), dict(bt=None),
               dict(sl=None), dict(out=None), dict(ws=None), dict(q=at + 8), dict(out=at + 8), dict(mb=at + 2),
               dict(of=at + 1), dict(ws=at + 16), dict(ks=at, vs=at)):
        assert _raw_prefix(make(), **kw) == INVALID, kw
    plan = make()
    assert _raw_prefix(plan, nb=int(plan.workspace_bytes) - 1) == SMALL
    for change in (lambda p: setattr(p, "prefixes", 2), lambda p: setattr(p.own, "q_len", 3),
                   lambda p: setattr(p.own.problem, "Hkv", 4), lambda p: setattr(p.own.problem, "out_dtype", _lib.FD_BF16),
                   lambda p: setattr(p, "ws_own_lse", 0), lambda p: setattr(p, "ws_own", p.ws_own + 16),
                   lambda p: setattr(p, "ws_shared", p.ws_own), lambda p: setattr(p, "workspace_bytes", p.ws_shared),
                   lambda p: setattr(p.shared, "seqs", 1)):
        bad = make()
        change(bad)
        assert _raw_prefix(bad) == INVALID
    cross = _lib.fd_plan_cross(problem(), [30, 30], num_sms=152)
    bad = make()
    bad.shared = cross
    assert _raw_prefix(bad) == INVALID


def _cross_tensors():
    bf = dict(dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    return dict(q=torch.zeros(4, 3, 8, 128, **bf), k_pages=torch.zeros(64, 16, 2, 128, **bf),
                v_pages=torch.zeros(64, 16, 2, 128, **bf), k_scale=None, v_scale=None,
                block_table=torch.zeros(2, 8, **i32), kv_lens=torch.zeros(2, **i32), out=torch.zeros(4, 3, 8, 128, **bf),
                lse=torch.zeros(4, 3, 8), workspace=torch.zeros(1 << 16, dtype=torch.uint8), q_lens=None, status=None)


@pytest.mark.parametrize("name,value", [
    ("q", None), ("q", torch.zeros(4, 3, 8, 128)), ("q", torch.zeros(4, 8, 128, dtype=torch.bfloat16)),
    ("q", torch.zeros(4, 3, 128, 8, dtype=torch.bfloat16).transpose(2, 3)),
    ("k_pages", torch.zeros(64, 16, 2, 64, dtype=torch.bfloat16)), ("k_scale", torch.zeros(64, 2)),
    ("block_table", torch.zeros(4, 8, dtype=torch.int32)), ("block_table", torch.zeros(2, 8)),
    ("kv_lens", torch.zeros(4, dtype=torch.int32)), ("q_lens", torch.zeros(2, dtype=torch.int32)),
    ("q_lens", torch.zeros(4, dtype=torch.int64)), ("out", torch.zeros(4, 3, 8, 128)),
    ("out", torch.zeros(4, 3, 8, 256, dtype=torch.bfloat16)[..., ::2]), ("lse", torch.zeros(4, 3, 8, dtype=torch.float64)),
    ("workspace", torch.zeros(16, dtype=torch.uint8)), ("status", torch.zeros(1)),
])
def test_cross_binding_names_the_argument(name, value):
    plan = _lib.fd_plan_cross(problem(), [100, 20], tokens=3, beams=2, num_sms=152)
    a = _cross_tensors()
    a[name] = value
    with pytest.raises(ValueError, match=name):
        _lib.fd_cross_paged(plan, **a)


def test_host_tensors_are_refused():
    plan = _lib.fd_plan_cross(problem(), [100, 20], tokens=3, beams=2, num_sms=152)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        _lib.fd_cross_paged(plan, **_cross_tensors())


def test_decoders_check_their_shapes():
    t = _cross_tensors()
    with pytest.raises(ValueError):
        fd.CrossDecoder.for_pools(t["q"], t["k_pages"], t["v_pages"], t["block_table"], [1, 2], beams=3, num_sms=152)
    with pytest.raises(ValueError):
        fd.CrossDecoder.for_pools(t["q"][0, 0], t["k_pages"], t["v_pages"], t["block_table"], [1, 2], num_sms=152)
    with pytest.raises(ValueError):
        fd.CrossDecoder.for_pools(t["q"][..., :64], t["k_pages"], t["v_pages"], t["block_table"], [1, 2], beams=2,
                                  num_sms=152)
    dec = fd.CrossDecoder.for_pools(t["q"], t["k_pages"], t["v_pages"], t["block_table"], [1, 2], beams=2, num_sms=152)
    assert dec.plan.tokens == 3 and dec.plan.seqs == 4
    pt = torch.zeros(3, 5, dtype=torch.int32)
    make = lambda of: fd.PrefixDecoder.for_pools(t["q"][:, 0], t["k_pages"], t["v_pages"], pt, [70, 3, 9], of,  # noqa: E731
                                                 torch.zeros(4, 8, dtype=torch.int32), [1, 2, 3, 4], num_sms=152)
    dec = make([2, -1, 0, 2])
    assert dec.members.tolist() == [2, 0, 3, 1] and dec.offsets.tolist() == [0, 1, 1, 3]
    dec.regroup([1, 1, 1, 1])
    assert dec.members.tolist() == [0, 1, 2, 3] and dec.offsets.tolist() == [0, 0, 4, 4]
    for bad in ([3, 0, 0, 0], [-2, 0, 0, 0], [0, 0, 0], [0.5, 0, 0, 0]):
        with pytest.raises(ValueError):
            make(bad)

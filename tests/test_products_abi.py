"""The grouped products' argument checks, made without a GPU: every refused call
names its fault and enqueues nothing."""

import ctypes

import pytest

from tests._lib import load

zr = load()
torch = pytest.importorskip("torch")

lib = zr._lib
A = 0x10000         # an address that no refused call reads
CALLS = [lib.zr_linear_forward, lib.zr_linear_input_grad]


def _plan():
    # weights 8 x 6 (params 1 and 2), another shape's param 3, another group's 4
    return zr.zr_plan_buckets([5, 48, 48, 40, 48], [0, 0, 0, 0, 1], [(2, 1), (1, 1)], 1000)


def _call(fn, **change):
    plan = _plan()
    v = dict(plan=plan.handle, params=(1, 2), counts=(3, 4), n=None, n_out=8, n_in=6, in_major=0, parts=(A, A),
             x=A, rows=7, x_stride=8, y=A, dtype=zr.ZR_FP32, y_stride=8, workspace=None, bytes=0, stream=None)
    v.update(change)
    for name, kind in (("params", ctypes.c_int64), ("counts", ctypes.c_int64), ("parts", ctypes.c_void_p)):
        if v[name] is not None:
            n = len(v[name])
            v[name] = (kind * max(n, 1))(*v[name])
            if name == "params" and v["n"] is None:
                v["n"] = n
    return fn(*v.values())


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("change,words", [
    (dict(plan=None), "plan"), (dict(n=-1), "n must"), (dict(params=None, n=2), "null param"),
    (dict(counts=None), "null param"), (dict(params=(1, 5)), "param id"), (dict(params=(-1, 1)), "param id"),
    (dict(params=(1, 4)), "share a group"), (dict(params=(1, 3)), "n_out * n_in"), (dict(n_out=0), "n_out and n_in"),
    (dict(n_in=-6), "n_out and n_in"), (dict(n_in=7), "n_out * n_in"), (dict(counts=(3, -1)), "negative"),
    (dict(counts=(3, 5)), "add up"), (dict(rows=-1), "rows must"), (dict(rows=6), "add up"),
    (dict(x_stride=5), "stride"), (dict(y_stride=5), "stride"), (dict(dtype=3), "dtype"),
    (dict(x=None), "input is null"), (dict(x=A + 1), "input is null"), (dict(y=None), "output is null"),
    (dict(y=A + 2), "output is null"), (dict(parts=None), "partition list"), (dict(parts=(A, None)), "partition 1"),
    (dict(parts=(A + 1, A)), "partition 0"),
])
def test_refusals(fn, change, words):
    assert _call(fn, **change) == zr.ZR_ERR_INVALID and words in zr.zr_last_error()


@pytest.mark.parametrize("fn", CALLS)
def test_unsupported(fn):
    plan = zr.zr_plan_buckets([1 << 23, 1 << 22], [0, 0], [(1, 1)], 1 << 30)
    base = dict(plan=plan.handle, params=(0,), counts=(1,), parts=(A,), rows=1 << 40, x_stride=1 << 23,
                y_stride=1 << 23)
    for change, words in ((dict(n_out=1 << 22, n_in=2), "n_out or n_in of"), (dict(n_out=2, n_in=1 << 22), "n_out or n_in"),
                          (dict(n_out=1 << 21, n_in=4), "input stride"),
                          (dict(n_out=1 << 21, n_in=4, counts=(1 << 31,)), "2^31 rows"),
                          (dict(n_out=1 << 21, n_in=4, counts=((1 << 31) - 1,)), "more tiles")):
        assert _call(fn, **{**base, **change}) == zr.ZR_ERR_UNSUPPORTED and words in zr.zr_last_error()


@pytest.mark.parametrize("fn", CALLS)
def test_nothing_to_do_needs_no_gpu(fn):
    assert _call(fn, counts=(0, 0), x=None, y=None, parts=None) == zr.ZR_OK
    assert _call(fn, params=(), counts=(), x=None, y=None, parts=None, rows=0) == zr.ZR_OK


def test_workspace():
    plan = zr.zr_plan_buckets([4096 * 4096], [0], [(1, 1)], 1 << 30)
    for call in (zr.zr_linear_forward_workspace, zr.zr_linear_input_grad_workspace):
        assert call(plan, [0], [0], 4096, 4096) == 0 and call(plan, [], [], 4096, 4096) == 0
        assert call(plan, [0], [4], 4096, 4096) > 0
        for bad in (([0], [-1], 4096, 4096), ([1], [1], 4096, 4096), ([0], [1], 4096, 4095), ([0], [1], 0, 0)):
            with pytest.raises(zr.ZrError):
                call(plan, *bad)
        with pytest.raises(zr.ZrError, match="counts has 1"):
            call(plan, [0, 0], [1], 4096, 4096)
        with pytest.raises(zr.ZrError, match="integers"):
            call(plan, [0], [1.5], 4096, 4096)
    assert lib.zr_linear_forward_workspace(plan.handle, None, None, 0, 1, 1, 0, None) == zr.ZR_ERR_INVALID


@pytest.mark.parametrize("fn", CALLS)
def test_workspace_refusals(fn):
    plan = zr.zr_plan_buckets([4096 * 4096], [0], [(1, 1)], 1 << 30)
    base = dict(plan=plan.handle, params=(0,), counts=(4,), n_out=4096, n_in=4096, parts=(A,), rows=4, x_stride=4096,
                y_stride=4096)
    for change in (dict(), dict(workspace=A, bytes=16), dict(workspace=A + 8, bytes=1 << 30)):
        assert _call(fn, **{**base, **change}) == zr.ZR_ERR_INVALID and "workspace" in zr.zr_last_error()


def test_host_tensors_are_refused():
    plan = _plan()
    x = torch.zeros(7, 6, dtype=torch.bfloat16)
    with pytest.raises(zr.ZrError):
        zr.zr_linear_forward(plan, [1, 2], [3, 4], [None, None], x, torch.zeros(7, 8))

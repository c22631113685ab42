"""The layer operators' argument checks, made without a GPU: every refused
call names its fault and enqueues nothing."""

import ctypes

import pytest

from tests._lib import load

zr = load()
torch = pytest.importorskip("torch")

lib = zr._lib
A = 0x10000         # an address that no refused call reads


def _plan(world=2):
    # table 10 x 6 (param 1), weight 4 x 8 (param 2), another group's param 3
    return zr.zr_plan_buckets([5, 60, 32, 12], [0, 0, 0, 1], [(world, 1), (2, 1)], 1000)


def _refused(status, message, *words):
    assert status == zr.ZR_ERR_INVALID or status == zr.ZR_ERR_UNSUPPORTED
    assert any(w in zr.zr_last_error() for w in words), zr.zr_last_error()


def test_layout():
    assert zr.zr_act_layout(1) == (32, 1) and zr.zr_act_layout(33) == (64, 2)
    assert zr.zr_act_layout(4096) == (4096, 128)
    for cols in (0, -1, 1 << 30):
        with pytest.raises(zr.ZrError):
            zr.zr_act_layout(cols)
    codes, scales = zr.act_empty(3, 33, "cpu")
    assert codes.shape == (3, 64) and codes.dtype is torch.float8_e4m3fn
    assert scales.shape == (3, 2) and scales.dtype is torch.uint8


@pytest.mark.parametrize("change,words", [
    (dict(plan=None), "plan"), (dict(param=-1), "param"), (dict(param=4), "param"),
    (dict(dim=0), "dim"), (dict(dim=7), "dim"), (dict(dtype=5), "dtype"), (dict(n=-1), "n must"),
    (dict(token_type=2), "token type"), (dict(tokens=None), "tokens"), (dict(tokens=A + 4), "tokens"),
    (dict(out=None), "out"), (dict(out=A + 1), "out"), (dict(stride=5), "out_stride"),
    (dict(parts=None), "parts"), (dict(parts=(A, None)), "partition 1"),
    (dict(parts=(A + 2, A)), "partition 0"),
])
def test_lookup_refusals(change, words):
    plan = _plan()
    v = dict(plan=plan.handle, param=1, dim=6, parts=(A, A), dtype=zr.ZR_FP32, tokens=A,
             token_type=zr.ZR_I64, n=3, out=A, stride=6)
    v.update(change)
    parts = None if v["parts"] is None else (ctypes.c_void_p * 2)(*v["parts"])
    st = lib.zr_embedding_lookup(v["plan"], v["param"], v["dim"], parts, v["dtype"], v["tokens"],
                                 v["token_type"], v["n"], 1.0, v["out"], v["stride"], None)
    assert st == zr.ZR_ERR_INVALID and words in zr.zr_last_error()


def test_lookup_of_nothing_needs_no_gpu():
    plan = _plan()
    parts = (ctypes.c_void_p * 2)(A, A)
    assert lib.zr_embedding_lookup(plan.handle, 1, 6, parts, zr.ZR_BF16, None, zr.ZR_I32, 0, 1.0,
                                   None, 6, None) == zr.ZR_OK


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("change,words", [
    (dict(plan=None), "plan"), (dict(param=9), "param"), (dict(dim=0), "dim"),
    (dict(dim=61), "dim"), (dict(n=-3), "n must"), (dict(n=1 << 31), "tokens or more"),
    (dict(tokens=None), "tokens"), (dict(token_type=-1), "token type"), (dict(dy=None), "dy"),
    (dict(dy=A + 2), "dy"), (dict(dtype=3), "dtype"), (dict(stride=5), "dy_stride"),
    (dict(grad=None), "main_grad"), (dict(grad=A + 1), "main_grad"), (dict(base=-1), "window"),
    (dict(length=-1), "window"), (dict(base=50, length=60), "window"),
    (dict(base=1 << 62, length=1 << 62), "window"),
    (dict(ws=None), "workspace"), (dict(ws=A + 8), "workspace"), (dict(ws_bytes=64), "workspace"),
])
def test_embedding_gradient_refusals(first, change, words):
    plan = _plan()
    v = dict(plan=plan.handle, param=1, dim=6, tokens=A, token_type=zr.ZR_I64, n=3, dy=A,
             dtype=zr.ZR_FP32, stride=6, grad=A, base=0, length=90, ws=A, ws_bytes=1 << 20)
    v.update(change)
    fn = lib.zr_ipg_accumulate_embedding_first if first else lib.zr_ipg_accumulate_embedding
    st = fn(v["plan"], v["param"], v["dim"], v["tokens"], v["token_type"], v["n"], 1.0, v["dy"],
            v["dtype"], v["stride"], v["grad"], v["base"], v["length"], v["ws"], v["ws_bytes"], None)
    assert st in (zr.ZR_ERR_INVALID, zr.ZR_ERR_UNSUPPORTED) and words in zr.zr_last_error()


def test_embedding_gradient_outside_the_window_needs_no_gpu():
    plan = _plan()
    for fn in (lib.zr_ipg_accumulate_embedding_first, lib.zr_ipg_accumulate_embedding):
        assert fn(plan.handle, 1, 6, A, zr.ZR_I64, 3, 1.0, A, zr.ZR_FP32, 6, A, 65, 33, A, 1 << 20,
                  None) == zr.ZR_OK
    assert lib.zr_ipg_accumulate_embedding(plan.handle, 1, 6, None, zr.ZR_I64, 0, 1.0, None,
                                           zr.ZR_FP32, 6, A, 0, 90, A, 1 << 20, None) == zr.ZR_OK


def test_calls_of_more_threads_than_a_launch_holds():
    """A launch holds fewer than 2^32 threads along an axis."""
    plan = _plan()
    parts = (ctypes.c_void_p * 2)(A, A)
    for n in (1 << 27, 1 << 28):
        assert lib.zr_embedding_lookup(plan.handle, 1, 6, parts, zr.ZR_BF16, A, zr.ZR_I32, n, 1.0,
                                       A, 6, None) == zr.ZR_ERR_UNSUPPORTED
    for fn in (lib.zr_ipg_accumulate_embedding_first, lib.zr_ipg_accumulate_embedding):
        assert fn(plan.handle, 1, 6, A, zr.ZR_I64, 1 << 28, 1.0, A, zr.ZR_FP32, 6, A, 0, 90, A,
                  1 << 60, None) == zr.ZR_ERR_UNSUPPORTED
    rows = 1 << 30      # of 32 columns, four threads a row
    assert lib.zr_act_quantize(A, zr.ZR_FP32, rows, 32, 32, A, A, None) == zr.ZR_ERR_UNSUPPORTED
    assert lib.zr_act_dequantize(A, A, rows, 32, A, zr.ZR_BF16, 32, None) == zr.ZR_ERR_UNSUPPORTED


def test_workspace_queries():
    plan = _plan()
    small = zr.zr_ipg_embedding_workspace(plan, 1, 6, 1, 0, 90)
    large = zr.zr_ipg_embedding_workspace(plan, 1, 6, 100000, 0, 90)
    assert 0 < small < large
    with pytest.raises(zr.ZrError, match="param"):
        zr.zr_ipg_embedding_workspace(plan, 4, 6, 1, 0, 90)
    with pytest.raises(zr.ZrError, match="window"):
        zr.zr_ipg_embedding_workspace(plan, 1, 6, 1, 0, 1000)
    assert lib.zr_ipg_embedding_workspace(plan.handle, 1, 6, 1, 0, 90, None) == zr.ZR_ERR_INVALID
    assert lib.zr_ipg_linear_workspace(plan.handle, None, 0, 0, 90, None) == zr.ZR_ERR_INVALID


@pytest.mark.parametrize("change,words", [
    (dict(x=None), "x is null"), (dict(x=A + 1), "x is null"), (dict(dtype=7), "dtype"),
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(cols=1 << 30, stride=1 << 30), "2^30"),
    (dict(stride=9), "stride"), (dict(codes=None), "codes"), (dict(codes=A + 8), "codes"),
    (dict(scales=None), "scales"), (dict(rows=1 << 62), "too many"),
])
def test_checkpoint_refusals(change, words):
    v = dict(x=A, dtype=zr.ZR_BF16, rows=4, cols=10, stride=10, codes=A, scales=A)
    v.update(change)
    st = lib.zr_act_quantize(v["x"], v["dtype"], v["rows"], v["cols"], v["stride"], v["codes"],
                             v["scales"], None)
    assert st in (zr.ZR_ERR_INVALID, zr.ZR_ERR_UNSUPPORTED) and words in zr.zr_last_error()
    words = words.replace("x is null", "out is null")
    st = lib.zr_act_dequantize(v["codes"], v["scales"], v["rows"], v["cols"], v["x"], v["dtype"],
                               v["stride"], None)
    assert st in (zr.ZR_ERR_INVALID, zr.ZR_ERR_UNSUPPORTED) and words in zr.zr_last_error()


def test_checkpoint_of_no_rows_needs_no_gpu():
    assert lib.zr_act_quantize(None, zr.ZR_FP32, 0, 10, 10, None, None, None) == zr.ZR_OK
    assert lib.zr_act_dequantize(None, None, 0, 10, None, zr.ZR_BF16, 10, None) == zr.ZR_OK


def _item(**change):
    v = dict(param=2, n_out=4, n_in=8, tokens=3, dy=A, dy_stride=4, codes=A, scales=A, in_major=0)
    v.update(change)
    return zr.zr_linear_grad(*v.values())


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("items,call,words", [
    ([_item(tokens=1 << 31)], {}, "2^31"), ([_item(dy_stride=1 << 24)], {}, "2^24"),
    ([_item(param=4)], {}, "param id"), ([_item(param=-1)], {}, "param id"),
    ([_item(), _item()], {}, "twice"),
    ([_item(), _item(param=3, n_out=3, n_in=4)], {}, "share a group"),
    ([_item(n_out=8)], {}, "n_out * n_in"), ([_item(n_out=0)], {}, "n_out * n_in"),
    ([_item(n_in=0)], {}, "n_out * n_in"), ([_item(tokens=-1)], {}, "rows"),
    ([_item(dy=None)], {}, "dy"), ([_item(dy=A + 1)], {}, "dy"),
    ([_item(dy_stride=3)], {}, "dy_stride"), ([_item(codes=None)], {}, "codes"),
    ([_item(codes=A + 4)], {}, "codes"), ([_item(scales=None)], {}, "scales"),
    ([_item()], dict(n=-1), "n must"), (None, dict(n=1), "null item"),
    ([_item()], dict(plan=None), "plan"), ([_item()], dict(grad=None), "main_grad"),
    ([_item()], dict(base=4, length=98), "window"), ([_item()], dict(base=-1), "window"),
])
def test_linear_gradient_refusals(first, items, call, words):
    plan = _plan()
    v = dict(plan=plan.handle, n=len(items or []), grad=A, base=0, length=98)
    v.update(call)
    arr = (zr.zr_linear_grad * len(items))(*items) if items else None
    fn = lib.zr_ipg_accumulate_linear_first if first else lib.zr_ipg_accumulate_linear
    st = fn(v["plan"], arr, v["n"], v["grad"], v["base"], v["length"], A, 1 << 30, None)
    assert st in (zr.ZR_ERR_INVALID, zr.ZR_ERR_UNSUPPORTED) and words in zr.zr_last_error()


def test_linear_gradient_of_more_threads_than_a_launch_holds():
    """512 a tile of 256 x 256 weights: 2^23 tiles are refused, of one weight or
    of several in a launch."""
    for numels, shapes in (([1 << 40], [(1 << 20, 1 << 20)]),
                           ([1 << 38] * 2, [(1 << 19, 1 << 19)] * 2)):
        plan = zr.zr_plan_buckets(numels, [0] * len(numels), [(1, 1)], 1 << 50)
        arr = (zr.zr_linear_grad * len(shapes))(*[
            _item(param=k, n_out=o, n_in=i, dy_stride=o) for k, (o, i) in enumerate(shapes)])
        for fn in (lib.zr_ipg_accumulate_linear_first, lib.zr_ipg_accumulate_linear):
            assert fn(plan.handle, arr, len(shapes), A, 0, sum(numels), A, 1 << 40,
                      None) == zr.ZR_ERR_UNSUPPORTED
            assert "too large" in zr.zr_last_error()
        out = ctypes.c_int64()
        assert lib.zr_ipg_linear_workspace(plan.handle, arr, len(shapes), 0, sum(numels),
                                           ctypes.byref(out)) == zr.ZR_ERR_UNSUPPORTED


def test_linear_workspace_depends_on_sizes_alone():
    """Neither on where dY lies nor on layers without tokens."""
    plan = zr.zr_plan_buckets([512 * 640, 640 * 512], [0, 0], [(1, 1)], 1 << 40)

    def need(*changes):
        v = [dict(param=0, n_out=512, n_in=640, dy_stride=512, tokens=2048),
             dict(param=1, n_out=640, n_in=512, dy_stride=640, tokens=2048)][:len(changes)]
        arr = (zr.zr_linear_grad * len(v))(*[_item(**{**a, **c}) for a, c in zip(v, changes)])
        out = ctypes.c_int64()
        assert lib.zr_ipg_linear_workspace(plan.handle, arr, len(v), 0, 2 * 512 * 640,
                                           ctypes.byref(out)) == zr.ZR_OK
        return out.value

    both = need({}, {})
    assert both > 0
    for dy, stride in ((A + 2, 640), (A, 641), (A + 14, 648)):
        assert need({}, dict(dy=dy, dy_stride=stride)) == both
    assert need({}, dict(tokens=0, dy=None, codes=None, scales=None)) == need({}) > 0


def test_linear_gradient_of_nothing_needs_no_gpu():
    plan = _plan()
    arr = (zr.zr_linear_grad * 1)(_item(tokens=0, dy=None, codes=None, scales=None))
    assert lib.zr_ipg_accumulate_linear(plan.handle, arr, 1, A, 0, 98, None, 0, None) == zr.ZR_OK
    assert lib.zr_ipg_accumulate_linear_first(plan.handle, None, 0, A, 0, 98, None, 0, None) == zr.ZR_OK
    # the weight lies behind the window
    arr = (zr.zr_linear_grad * 1)(_item())
    assert lib.zr_ipg_accumulate_linear_first(plan.handle, arr, 1, A, 0, 65, A, 1 << 20, None) == zr.ZR_OK


def test_binding_refuses_host_tensors_shapes_and_types():
    plan = _plan()
    dy, grad = torch.zeros(3, 6), torch.zeros(90)
    ws = torch.zeros(4096, dtype=torch.uint8)
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(zr.ZrError, match="device tensor"):
        zr.zr_ipg_accumulate_embedding(plan, 1, 6, ids, dy, grad, ws, stream=0)
    with pytest.raises(zr.ZrError, match="tokens must be"):
        zr.zr_embedding_lookup(plan, 1, 6, [grad, grad], ids.float(), dy, stream=0)
    with pytest.raises(zr.ZrError, match="x must be one of"):
        zr.zr_act_quantize(dy.half(), *zr.act_empty(3, 6, "cpu"), stream=0)
    with pytest.raises(zr.ZrError, match="x has shape"):
        zr.zr_act_quantize(dy[0], *zr.act_empty(3, 6, "cpu"), stream=0)
    with pytest.raises(zr.ZrError, match="dy must be one of"):
        zr.zr_ipg_accumulate_linear(plan, [(2, dy, *zr.act_empty(3, 8, "cpu"))], grad, ws, stream=0)

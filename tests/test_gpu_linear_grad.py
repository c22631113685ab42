"""zr_ipg_accumulate_linear against the float64 oracle: sizes around the tiles'
edges, windows that cut the weight, lists of layers, both storage orders."""

import numpy as np
import pytest

from oracle.layers import dequantize_oracle, linear_grad_oracle, quantize_oracle
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._layers import Window, check_window, checkpoint, rows, workspace  # noqa: E402

SIZES = [  # outputs, inputs, tokens
    (1, 1, 1), (7, 5, 3), (128, 128, 64), (130, 97, 65), (300, 70, 63), (64, 513, 17),
    (257, 256, 300), (96, 40, 0), (1000, 33, 129), (33, 1000, 16), (640, 384, 1025), (2, 3, 5000),
    (129, 127, 4100), (513, 511, 7), (264, 512, 4096), (512, 264, 3001), (8, 40, 191),
    (776, 300, 128),
]


def _layer(rng, n_out, n_in, tokens, pad=0, whole=False):
    """dY and a checkpoint, as device tensors and as float64 values.  whole:
    small whole numbers, whose sums are exact in fp32."""
    if whole:
        x = rng.integers(-8, 9, (tokens, n_in)).astype(np.float32)
        dy = rng.integers(-8, 9, (tokens, n_out)).astype(np.float32)
    else:
        x = rng.standard_normal((tokens, n_in)) * np.exp(rng.standard_normal(n_in))
        dy = rng.standard_normal((tokens, n_out))
    codes, scales = quantize_oracle(x.astype(np.float32))
    t, held = rows(dy, True, pad, 1 if pad else 0)
    return (t, *checkpoint(codes, scales)), held, dequantize_oracle(codes, scales, n_in)


def _run(plan, items, win, base, first, stream=None):
    ws = workspace(zr.zr_ipg_linear_workspace(plan, items, base, win.grad.numel()))
    call = zr.zr_ipg_accumulate_linear_first if first else zr.zr_ipg_accumulate_linear
    call(plan, items, win.grad, ws, window_base=base, stream=stream)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("in_major", [False, True])
@pytest.mark.parametrize("n_out,n_in,tokens", SIZES)
def test_gradient(n_out, n_in, tokens, in_major, first):
    rng = np.random.default_rng(n_out * 7 + n_in + tokens)
    lead = 5
    for whole, pad, world in ((True, 0, 1), (False, 3, 1), (False, 0, 3)):
        plan = zr.zr_plan_buckets([lead, n_out * n_in, 11], [0] * 3, [(world, 1)], 1 << 40)
        P = zr.zr_plan_group_info(plan, 0)[2]
        item, dy, x = _layer(rng, n_out, n_in, tokens, pad, whole)
        g, size = linear_grad_oracle(dy, x, in_major)
        for part in range(world):
            win = Window(P, part, offset=part % 4)
            _run(plan, [(1, *item, in_major)], win, part * P, first)
            check_window(win, lead - part * P, g, np.zeros_like(size) if whole else size, tokens,
                         first, None if first or tokens else False, f"part {part} of {world}")


@pytest.mark.parametrize("in_major", [False, True])
def test_windows_that_cut_rows(in_major):
    """Windows that start and end inside a row, hold one row, one element or
    nothing of the weight."""
    rng = np.random.default_rng(4)
    n_out, n_in, tokens = 200, 150, 40
    plan = zr.zr_plan_buckets([9, n_out * n_in, 50], [0] * 3, [(1, 1)], 1 << 40)
    item, dy, x = _layer(rng, n_out, n_in, tokens)
    g, size = linear_grad_oracle(dy, x, in_major)
    for base, length in ((0, 9), (3, 10), (9, 1), (160, 3), (9 + 150 * 7, 150), (9 + 133, 20000),
                         (9 + 200 * 128 - 1, 2), (30000, 9), (30009, 50), (1, 30058), (500, 0)):
        win = Window(length, base)
        _run(plan, [(1, *item, in_major)], win, base, False)
        check_window(win, 9 - base, g, size, tokens, False, None, f"window {base}+{length}")


def test_many_layers_in_one_call():
    """Forty layers, some without tokens, two of them on one checkpoint."""
    rng = np.random.default_rng(6)
    shapes = [(int(rng.integers(1, 300)), int(rng.integers(1, 300)), int(rng.integers(0, 200)))
              for _ in range(40)]
    shapes[3] = (shapes[3][0], 64, 77)
    shapes[4] = (shapes[4][0], 64, 77)
    shapes[7] = (*shapes[7][:2], 0)
    plan = zr.zr_plan_buckets([a * b for a, b, _ in shapes], [0] * 40, [(1, 1)], 1 << 40)
    layers = [_layer(rng, *s) for s in shapes]
    layers[4] = ((layers[4][0][0], *layers[3][0][1:]), layers[4][1], layers[3][2])
    total = sum(a * b for a, b, _ in shapes)
    for first in (True, False):
        win = Window(total, 1)
        items = [(k, *item, k % 2 == 1) for k, (item, _, _) in enumerate(layers)]
        _run(plan, items[::-1], win, 0, first)
        grads = [linear_grad_oracle(dy, x, k % 2 == 1) for k, (_, dy, x) in enumerate(layers)]
        terms = np.concatenate([np.full(a * b, t) for a, b, t in shapes])
        check_window(win, 0, np.concatenate([g.ravel() for g, _ in grads]),
                     np.concatenate([s.ravel() for _, s in grads]), terms, first,
                     None if first else terms > 0)


def test_long_sums_and_few_weights():
    rng = np.random.default_rng(11)
    for n_out, n_in, tokens in ((60, 50, 20000), (300, 200, 9000)):
        plan = zr.zr_plan_buckets([n_out * n_in], [0], [(1, 1)], 1 << 40)
        for whole in (True, False):
            item, dy, x = _layer(rng, n_out, n_in, tokens, whole=whole)
            g, size = linear_grad_oracle(dy, x, False)
            assert np.abs(g).max() < 2 ** 24
            for first in (False, True):
                win = Window(n_out * n_in, 3)
                _run(plan, [(0, *item)], win, 0, first)
                check_window(win, 0, g, np.zeros_like(size) if whole else size, tokens, first)


@pytest.mark.parametrize("in_major", [False, True])
def test_rows_of_dy_on_and_off_sixteen_bytes_in_one_call(in_major):
    """Layers of both kinds, and a weight cut along its tokens among them."""
    rng = np.random.default_rng(21)
    shapes = [(256, 130, 4500, 0), (256, 130, 4500, 1), (40, 70, 600, 8), (41, 70, 600, 0)]
    plan = zr.zr_plan_buckets([a * b for a, b, _, _ in shapes], [0] * 4, [(1, 1)], 1 << 40)
    layers = [_layer(rng, a, b, t, pad, whole=True) for a, b, t, pad in shapes]
    grads = [linear_grad_oracle(dy, x, in_major)[0] for _, dy, x in layers]
    for first in (False, True):
        win = Window(sum(a * b for a, b, _, _ in shapes), 1)
        _run(plan, [(k, *item, in_major) for k, (item, _, _) in enumerate(layers)], win, 0, first)
        g = np.concatenate([g.ravel() for g in grads])
        check_window(win, 0, g, np.zeros_like(g), 4500, first)


def test_small_and_large_scales():
    """Blocks at the ends of the scale bytes' range: every operand is a
    normal bf16 number, and so is every product in fp32."""
    rng = np.random.default_rng(12)
    x = rng.standard_normal((96, 64))
    x[:48] *= 2.0 ** -100
    x[48:] *= 2.0 ** 100
    for part, dscale in ((slice(0, 48), 2.0 ** 20), (slice(48, 96), 2.0 ** -80)):
        codes, scales = quantize_oracle(x[part].astype(np.float32))
        t, dy = rows(rng.standard_normal((48, 40)) * dscale, True)
        plan = zr.zr_plan_buckets([40 * 64], [0], [(1, 1)], 1 << 40)
        win = Window(40 * 64, 3)
        _run(plan, [(0, t, *checkpoint(codes, scales))], win, 0, True)
        g, size = linear_grad_oracle(dy, dequantize_oracle(codes, scales, 64), False)
        check_window(win, 0, g, size, 48, True)


@pytest.mark.parametrize("dy,x,want", [
    (2.0 ** -133, 2.0 ** 110, 2.0 ** -21),      # the least bf16 number
    (2.0 ** -60, 2.0 ** -88, 2.0 ** -146),      # a subnormal sum
    (2.0 ** -20, float.fromhex("0x1.fep127"), float("inf")),   # coded up to 2^128
])
def test_ends_of_the_number_range(dy, x, want):
    """Four equal products of powers of two: exact, subnormals included."""
    codes, scales = zr.act_empty(4, 32)
    zr.zr_act_quantize(torch.full((4, 32), x, device="cuda"), codes, scales)
    plan = zr.zr_plan_buckets([16 * 32], [0], [(1, 1)], 1 << 40)
    grad = torch.empty(512, device="cuda")
    item = (0, torch.full((4, 16), dy, device="cuda").bfloat16(), codes, scales)
    zr.zr_ipg_accumulate_linear_first(plan, [item], grad, None)
    assert (grad == want).all()


def test_a_nan_stays_in_its_row_and_column():
    rng = np.random.default_rng(13)
    item, dy, x = _layer(rng, 140, 70, 30)
    item[0][4, 9] = float("nan")
    plan = zr.zr_plan_buckets([140 * 70], [0], [(1, 1)], 1 << 40)
    win = Window(140 * 70, 3)
    _run(plan, [(0, *item)], win, 0, True)
    got = win.after().reshape(140, 70)
    assert np.isnan(got[9]).all() and np.isfinite(np.delete(got, 9, 0)).all()


def test_same_bits_on_every_run_and_on_another_stream():
    rng = np.random.default_rng(14)
    item, _, _ = _layer(rng, 200, 120, 3000)
    plan = zr.zr_plan_buckets([200 * 120], [0], [(1, 1)], 1 << 40)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for stream in (None, None, s):
        win = Window(200 * 120, 3)
        torch.cuda.synchronize()
        _run(plan, [(0, *item)], win, 0, True, stream)
        got.append(win.after())
    assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])


def test_captured_and_replayed():
    rng = np.random.default_rng(15)
    shapes = [(260, 140, 500), (30, 140, 500), (64, 64, 2000)]
    plan = zr.zr_plan_buckets([a * b for a, b, _ in shapes], [0] * 3, [(1, 1)], 1 << 40)
    layers = [[(k, *_layer(rng, *s)[0]) for k, s in enumerate(shapes)] for _ in range(2)]
    n = sum(a * b for a, b, _ in shapes)
    grad, want = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    ws = workspace(max(zr.zr_ipg_linear_workspace(plan, b, 0, n) for b in layers))

    def step(out):
        zr.zr_ipg_accumulate_linear_first(plan, layers[0], out, ws)
        zr.zr_ipg_accumulate_linear(plan, layers[1], out, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(grad)
    for r in range(4):
        for batch in layers:
            for item in batch:
                item[1].copy_(torch.randn(item[1].shape, device="cuda"))
        step(want)
        grad.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, want) and want.abs().max() > 1


def _bits(plan, items, length, first, before):
    """main_grad after one call on `before`, with NaN behind the _first form."""
    grad = torch.full((length,), float("nan"), device="cuda") if first else before.clone()
    ws = workspace(zr.zr_ipg_linear_workspace(plan, items, 0, length))
    (zr.zr_ipg_accumulate_linear_first if first else zr.zr_ipg_accumulate_linear)(plan, items, grad, ws)
    return grad


@pytest.mark.parametrize("in_major", [False, True])
def test_first_gives_the_bits_of_the_plain_form_on_zeros(in_major):
    """Also beside a layer without tokens, whose weights only the _first form
    writes: the other layer's sums are cut into the same pieces."""
    rng = np.random.default_rng(31)
    plan = zr.zr_plan_buckets([512 * 640, 640 * 512], [0, 0], [(1, 1)], 1 << 40)
    full, _, _ = _layer(rng, 512, 640, 2048)
    none, _, _ = _layer(rng, 640, 512, 0)
    items, n = [(0, *full, in_major), (1, *none, in_major)], 2 * 512 * 640
    first = _bits(plan, items, n, True, None)
    added = _bits(plan, items, n, False, torch.zeros(n, device="cuda"))
    assert torch.equal(first, added) and (first[n // 2:] == 0).all()
    # nor does the layer without tokens matter to the other one's sums
    alone = _bits(plan, items[:1], n, True, None)
    assert torch.equal(first[:n // 2], alone[:n // 2]) and alone[n // 2:].isnan().all()


@pytest.mark.parametrize("in_major", [False, True])
def test_bits_do_not_depend_on_where_dy_lies(in_major):
    """Layers' rows of dY on 16 bytes, off them, or some on and some off: the
    sums have the same order."""
    rng = np.random.default_rng(32)
    shapes = [(512, 640, 2048), (264, 512, 3001), (96, 300, 700)]
    plan = zr.zr_plan_buckets([a * b for a, b, _ in shapes], [0] * 3, [(1, 1)], 1 << 40)
    layers = [_layer(rng, *s)[0] for s in shapes]
    n = sum(a * b for a, b, _ in shapes)

    def off(dy):
        """The same rows, each 2 bytes off 16."""
        wide = torch.empty(dy.shape[0] * dy.shape[1] + 1, dtype=dy.dtype, device="cuda")[1:].view(dy.shape)
        return wide.copy_(dy)

    want, need = None, None
    for places in ((0, 0, 0), (1, 1, 1), (1, 0, 0), (0, 1, 0), (1, 0, 1)):
        items = [(k, off(dy) if p else dy, c, s, in_major)
                 for k, (p, (dy, c, s)) in enumerate(zip(places, layers))]
        got = _bits(plan, items, n, True, None)
        size = zr.zr_ipg_linear_workspace(plan, items, 0, n)
        want, need = (got, size) if want is None else (want, need)
        assert torch.equal(got, want) and size == need, places


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("in_major", [False, True])
@pytest.mark.parametrize("shapes", [
    [(4352, 4096, 640)],                                    # 272 tiles: 16 cut
    [(2048, 4096, 700), (2304, 4000, 643)],                 # the second partly whole, partly cut
    [(4100, 2050, 330), (515, 8200, 326), (2049, 260, 0)],  # 252 tiles and 18 without tokens
    [(9000, 520, 1300), (300, 33000, 60)],                  # more than a round whose tokens differ
])
def test_more_tiles_than_cus(shapes, in_major, first):
    """Whole numbers, whose sums are exact, in weights of several rounds of
    tiles; nothing is written behind the workspace."""
    gen = torch.Generator("cuda").manual_seed(len(shapes) * 10 + in_major)
    plan = zr.zr_plan_buckets([a * b for a, b, _ in shapes], [0] * len(shapes), [(1, 1)], 1 << 40)
    items, want = [], []
    for k, (n_out, n_in, tokens) in enumerate(shapes):
        dy = torch.randint(-8, 9, (tokens, n_out), device="cuda", generator=gen).bfloat16()
        x = torch.randint(-8, 9, (tokens, n_in), device="cuda", generator=gen).float()
        codes, scales = zr.act_empty(tokens, n_in)
        zr.zr_act_quantize(x, codes, scales)
        items.append((k, dy, codes, scales, in_major))
        a, b = (x.double(), dy.double()) if in_major else (dy.double(), x.double())
        want.append((a.t().contiguous() @ b).flatten())
    want = torch.cat(want).float()
    n = want.numel()
    grad = torch.full((n + 64,), 3.0, device="cuda")
    need = zr.zr_ipg_linear_workspace(plan, items, 0, n)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    call = zr.zr_ipg_accumulate_linear_first if first else zr.zr_ipg_accumulate_linear
    call(plan, items, grad[:n], ws[:need])
    assert torch.equal(grad[:n], want if first else want + 3.0)
    assert (grad[n:] == 3.0).all() and (ws[need:] == 0xA5).all()

"""zr_embedding_lookup and zr_ipg_accumulate_embedding against the float64
oracle, at the sizes, windows and ids where they can go wrong."""

import numpy as np
import pytest

from oracle.layers import embedding_grad_oracle, lookup_oracle
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._gpu import assert_bits_equal, host_f32, host_u16, to_dev  # noqa: E402
from tests._layers import Window, bf16_patterns, check_window, rows, workspace  # noqa: E402


def _plan(numels, world):
    return zr.zr_plan_buckets(numels, [0] * len(numels), [(world, 1)], 1 << 40)


def _ids(rng, vocab, n, masked=0.1):
    """Ids whose frequency falls with their rank; some outside the table."""
    t = np.minimum(np.exp(rng.random(n) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    out = rng.random(n) < masked
    t[out] = rng.choice([-100, -1, vocab, vocab + 5, 2 ** 31 - 1, -2 ** 31], int(out.sum()))
    return t


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,dim,world,lead,n,pad", [
    (1, 1, 1, 0, 1, 0), (5, 3, 4, 1, 7, 0), (50, 8, 8, 0, 33, 8), (11, 64, 3, 5, 1, 0),
    (7, 1001, 5, 2, 40, 3), (300, 256, 8, 64, 513, 0), (9, 2048, 2, 0, 5, 0),
    (6, 4100, 3, 7, 19, 1), (3, 8200, 64, 0, 4, 0), (40, 4096, 1, 0, 64, 0),
])
def test_lookup(vocab, dim, world, lead, n, pad, bf16):
    rng = np.random.default_rng(vocab * 1000 + dim)
    numels = ([lead] if lead else []) + [vocab * dim, 13]
    plan, param = _plan(numels, world), 1 if lead else 0
    P = zr.zr_plan_group_info(plan, 0)[2]
    flat = rng.standard_normal(P * world).astype(np.float32)
    stored = bf16_patterns(flat) if bf16 else flat
    parts = [to_dev(stored[k * P:(k + 1) * P], k % 3) for k in range(world)]
    for k in range(world):          # partitions without a row of the table
        if (k + 1) * P <= lead or k * P >= lead + vocab * dim:
            parts[k] = None
    t = _ids(rng, vocab, n)
    table = stored[lead:lead + vocab * dim].reshape(vocab, dim)
    for scale in (1.0, 0.3):
        for wide in (True, False):
            ids = torch.from_numpy(t if wide else t.astype(np.int32)).cuda()
            buf = torch.full((n * (dim + pad) + 8,), 7.5, dtype=torch.bfloat16 if bf16 else torch.float32,
                             device="cuda")
            out = buf[3:3 + n * (dim + pad)].view(n, dim + pad)[:, :dim]
            zr.zr_embedding_lookup(plan, param, dim, parts, ids, out, scale=scale)
            want = lookup_oracle(table, t, scale, bf16)
            if bf16:
                assert np.array_equal(host_u16(out.contiguous()), want)
            else:
                assert_bits_equal(host_f32(out.contiguous()), want, "rows")
            whole = buf.float().cpu().numpy()
            gaps = np.ones(whole.size, bool)
            for i in range(n):
                gaps[3 + i * (dim + pad):3 + i * (dim + pad) + dim] = False
            assert (whole[gaps] == 7.5).all(), "wrote between the rows"


def test_lookup_of_a_gathered_vector_and_of_nothing():
    plan = _plan([12 * 40], 4)
    flat = torch.randn(480, device="cuda")
    ids = torch.tensor([[3, 11], [0, 3]], dtype=torch.int32, device="cuda")
    out = torch.empty(4, 40, device="cuda")
    zr.zr_embedding_lookup(plan, 0, 40, list(flat.split(120)), ids, out)
    assert torch.equal(out, flat.view(12, 40)[ids.flatten().long()])
    zr.zr_embedding_lookup(plan, 0, 40, list(flat.split(120)), ids[:0], out[:0])


GRAD = [  # vocab, dim, world, lead, n
    (1, 1, 1, 0, 1), (5, 3, 2, 1, 9), (3, 4, 1, 0, 200), (40, 64, 3, 5, 65), (2000, 8, 8, 0, 1000),
    (7, 1001, 2, 2, 40), (300, 1024, 4, 64, 513), (9, 2050, 2, 0, 100), (50000, 2, 1, 3, 3000),
    (1, 260, 1, 0, 700), (1100, 33, 1, 0, 4097), (262143, 1, 1, 0, 3000), (600001, 2, 1, 3, 4000),
    (2, 5, 1, 0, 20001), (700, 3, 2, 1, 40001),
]


def _grad_case(vocab, dim, world, lead, n, bf16, first, part, t, dy, scale, pad=0, wide=True,
               exact=False, stream=None):
    numels = ([lead] if lead else []) + [vocab * dim, 13]
    plan, param = _plan(numels, world), 1 if lead else 0
    P = zr.zr_plan_group_info(plan, 0)[2]
    base, length = (part * P, P) if part is not None else (0, P * world)
    drows, held = rows(dy, bf16, pad, 1)
    ids = torch.from_numpy(t if wide else t.astype(np.int32)).cuda()
    win = Window(length, n)
    ws = workspace(zr.zr_ipg_embedding_workspace(plan, param, dim, n, base, length))
    call = zr.zr_ipg_accumulate_embedding_first if first else zr.zr_ipg_accumulate_embedding
    call(plan, param, dim, ids, drows, win.grad, ws, window_base=base, scale=scale, stream=stream)
    g, size, count = embedding_grad_oracle(vocab, t, held, scale)
    if exact:           # whole numbers whose sums fp32 holds: no rounding at all
        size = np.zeros_like(size)
    return check_window(win, lead - base, g, size, count[:, None] + 1, first,
                        None if first else count[:, None] > 0, f"part {part}")


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,dim,world,lead,n", GRAD)
def test_gradient(vocab, dim, world, lead, n, bf16, first):
    rng = np.random.default_rng(vocab + 7 * dim + n)
    t = _ids(rng, vocab, n)
    dy = rng.standard_normal((n, dim)).astype(np.float32)
    outside = (t < 0) | (t >= vocab)
    dy[outside] = rng.choice([np.nan, np.inf, -np.inf], (int(outside.sum()), 1))
    for part in [None] + list(range(world)):
        _grad_case(vocab, dim, world, lead, n, bf16, first, part, t, dy, 1.7,
                   pad=3 if part == 0 else 0, wide=part != 1)


@pytest.mark.parametrize("first", [False, True])
def test_gradient_of_whole_numbers_is_exact(first):
    """Sums of whole numbers below 2^24 round nowhere; the window's elements
    are the oracle's up to the last add's rounding."""
    rng = np.random.default_rng(5)
    for vocab, dim, n in ((70, 520, 3000), (4, 100, 5000), (1, 64, 10000)):
        t = _ids(rng, vocab, n)
        dy = rng.integers(-100, 101, (n, dim)).astype(np.float32)
        _grad_case(vocab, dim, 1, 0, n, True, first, None, t, dy, 2.0, exact=True)


@pytest.mark.parametrize("first", [False, True])
def test_gradient_without_a_valid_token(first):
    dy = np.full((50, 12), np.nan, np.float32)
    t = np.full(50, -100)
    _grad_case(9, 12, 2, 0, 50, False, first, None, t, dy, 1.0)
    _grad_case(9, 12, 2, 0, 0, False, first, 1, t[:0], dy[:0], 1.0)


def test_ids_at_the_ends_of_64_bits():
    t = np.array([-2 ** 63, 2 ** 63 - 1, 3, -2 ** 63 + 5, 2 ** 62, 2 ** 32 + 3])
    dy = np.full((6, 8), np.nan, np.float32)
    dy[2] = 2.0
    for part in (0, 1):
        _grad_case(9, 8, 2, 0, 6, False, True, part, t, dy, 1.0)
    plan, out = _plan([72], 1), torch.empty(6, 8, device="cuda")
    zr.zr_embedding_lookup(plan, 0, 8, [torch.ones(72, device="cuda")], torch.from_numpy(t).cuda(), out)
    assert out.sum(1).tolist() == [0, 0, 8, 0, 0, 0]


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("n", [700, 9000, 40000])
def test_gradient_of_ids_that_one_workgroup_sorts(n, first):
    """Ids a power of two apart, so that the rows dealt out to one workgroup
    meet within every 64 tokens; and batches longer than a wave keeps."""
    rng = np.random.default_rng(n)
    t = 256 * rng.integers(0, 60, n) + rng.integers(0, 2, n)
    t[::7] = rng.integers(0, 15500, t[::7].size)
    dy = rng.integers(-50, 51, (n, 12)).astype(np.float32)
    _grad_case(15500, 12, 1, 0, n, True, first, None, t, dy, 1.0, exact=True)


def test_gradient_has_the_same_bits_on_every_run():
    rng = np.random.default_rng(8)
    t = _ids(rng, 500, 20000)
    dy = rng.standard_normal((20000, 96)).astype(np.float32)
    a = _grad_case(500, 96, 1, 0, 20000, False, True, None, t, dy, 1.0)
    b = _grad_case(500, 96, 1, 0, 20000, False, True, None, t, dy, 1.0)
    assert np.array_equal(a, b)


def test_gradient_on_another_stream():
    rng = np.random.default_rng(9)
    t = _ids(rng, 60, 400)
    dy = rng.standard_normal((400, 70)).astype(np.float32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _grad_case(60, 70, 2, 3, 400, True, False, None, t, dy, 1.0, stream=s)


def test_gradient_captured_and_replayed():
    """Two micro-batches captured in one graph; the replays take new ids and
    gradients written into the captured buffers."""
    rng = np.random.default_rng(10)
    vocab, dim, n = 400, 130, 900
    plan = _plan([vocab * dim], 2)
    P = zr.zr_plan_group_info(plan, 0)[2]
    ids = [torch.zeros(n, dtype=torch.int64, device="cuda") for _ in range(2)]
    dy = [torch.zeros(n, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    grad, want = torch.zeros(P, device="cuda"), torch.zeros(P, device="cuda")
    ws = workspace(zr.zr_ipg_embedding_workspace(plan, 0, dim, n, P, P))

    def step(out):
        zr.zr_ipg_accumulate_embedding_first(plan, 0, dim, ids[0], dy[0], out, ws, window_base=P)
        zr.zr_ipg_accumulate_embedding(plan, 0, dim, ids[1], dy[1], out, ws, window_base=P)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(grad)
    for _ in range(4):
        for k in range(2):
            ids[k].copy_(torch.from_numpy(_ids(rng, vocab, n)))
            dy[k].copy_(torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)))
        step(want)
        grad.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, want) and want.abs().max() > 1


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dim", [1, 3, 7, 8, 130, 1001, 4101])
@pytest.mark.parametrize("scale", [-1.0, -0.0, float("inf"), float("nan")])
def test_lookup_of_padding_is_plus_zero_whatever_the_scale(scale, dim, bf16):
    """An id outside the table reads nothing and is scaled by nothing: +0 in
    rows of every width, beside rows of the table that the scale makes
    negative, infinite or NaN."""
    plan = _plan([5 * dim], 2)
    P = zr.zr_plan_group_info(plan, 0)[2]
    table = torch.rand(2 * P, device="cuda") + 0.5
    table = table.bfloat16() if bf16 else table
    ids = torch.tensor([-1, 3, 5, 0, 2 ** 62, 4, -2 ** 63], device="cuda")
    out = torch.full((7, dim), 7.5, dtype=table.dtype, device="cuda")
    zr.zr_embedding_lookup(plan, 0, dim, list(table.split(P)), ids, out, scale=scale)
    bits = out.view(torch.int16 if bf16 else torch.int32).cpu()
    assert (bits[[0, 2, 4, 6]] == 0).all()
    want = (table[:5 * dim].view(5, dim)[[3, 0, 4]].float() * scale).to(table.dtype)
    assert torch.equal(out[[1, 3, 5]].isnan(), want.isnan())
    assert np.isnan(scale) or torch.equal(out[[1, 3, 5]], want)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,dim,n", [(7, 4097, 40), (40, 4100, 300), (5, 8192, 200), (3, 8203, 70),
                                         (2, 20001, 30)])
def test_gradient_of_rows_wider_than_a_workgroup(vocab, dim, n, bf16, first):
    """Several workgroups share a row's columns; nothing is written behind the
    workspace."""
    rng = np.random.default_rng(vocab + dim)
    t = _ids(rng, vocab, n)
    dy = rng.integers(-50, 51, (n, dim)).astype(np.float32)
    dy[(t < 0) | (t >= vocab)] = np.nan
    for part in (None, 0, 1):
        _grad_case(vocab, dim, 2, 3, n, bf16, first, part, t, dy, 2.0, pad=part == 0, exact=True)
    plan = _plan([vocab * dim], 1)
    size = zr.zr_ipg_embedding_workspace(plan, 0, dim, n, 0, vocab * dim)
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    rows_, _ = rows(dy, bf16)
    zr.zr_ipg_accumulate_embedding_first(plan, 0, dim, torch.from_numpy(t).cuda(), rows_,
                                         torch.empty(vocab * dim, device="cuda"), ws[:size])
    assert (ws[size:] == 0xA5).all()


@pytest.mark.parametrize("vocab,dim,n", [(300, 96, 5000), (9, 1001, 700), (5000, 130, 900), (4, 3, 3000)])
def test_gradient_bits_do_not_depend_on_the_form_or_on_where_dy_lies(vocab, dim, n):
    rng = np.random.default_rng(n)
    plan, t = _plan([vocab * dim], 1), torch.from_numpy(_ids(rng, vocab, n)).cuda()
    values = rng.standard_normal((n, dim)).astype(np.float32)
    values[::3] *= -0.0
    ws = workspace(zr.zr_ipg_embedding_workspace(plan, 0, dim, n, 0, vocab * dim))
    for bf16 in (False, True):
        got = []
        for pad, offset in ((0, 0), (0, 1), (5, 3)):
            dy, _ = rows(values, bf16, pad, offset)
            grad = torch.full((vocab * dim,), float("nan"), device="cuda")
            zr.zr_ipg_accumulate_embedding_first(plan, 0, dim, t, dy, grad, ws, scale=-1.3)
            added = torch.zeros(vocab * dim, device="cuda")
            zr.zr_ipg_accumulate_embedding(plan, 0, dim, t, dy, added, ws, scale=-1.3)
            got += [host_f32(grad), host_f32(added)]
        for other in got[1:]:
            assert_bits_equal(other, got[0], "sums")

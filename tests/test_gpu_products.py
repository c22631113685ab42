"""The grouped products against numpy in 64 bits.

A sum of m products of bf16 values, exact in fp32, each add off by at most 2^-23
of its result (the matrix cores may truncate), is within m * 2^-23 * sum |term|
of the exact sum in any order; then the output's own rounding."""

import numpy as np
import pytest

from oracle.layers import bf16_widen_oracle
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._gpu import to_dev  # noqa: E402
from tests._layers import U, bf16_patterns, rows as device_rows, workspace  # noqa: E402


class Case:
    def __init__(self, seed, n_out, n_in, counts, input_grad, in_major=False, world=1, lead=0, align=1, bf16=True,
                 x_pad=0, y_pad=0, offset=0, behind=0, part_offset=0, params=None, whole=False):
        rng = np.random.default_rng(seed)
        numels = ([lead] if lead else []) + [n_out * n_in] * (len(counts) if params is None else max(params) + 1) + [7]
        self.plan = zr.zr_plan_buckets(numels, [0] * len(numels), [(world, 1)], 1 << 30, align=align)
        total, padded, P, _ = zr.zr_plan_group_info(self.plan, 0)
        flat = np.zeros(padded, np.float32)
        draw = (lambda *s: rng.integers(-4, 5, s)) if whole else (lambda *s: rng.standard_normal(s))
        flat[:total] = draw(total)
        bits = bf16_patterns(flat)
        self.flat = bf16_widen_oracle(bits).astype(np.float64)
        self.params = [k + bool(lead) for k in (range(len(counts)) if params is None else params)]
        self.counts, self.input_grad, self.in_major, self.bf16 = counts, input_grad, in_major, bf16
        offsets = [zr.zr_plan_param_offset(self.plan, p) for p in self.params]
        self.parts = []
        for k in range(world):
            used = any(c and o < (k + 1) * P and o + n_out * n_in > k * P for c, o in zip(counts, offsets))
            self.parts.append(to_dev(bits[k * P:(k + 1) * P], part_offset) if used else None)
        shape = (n_in, n_out) if in_major else (n_out, n_in)
        self.weights = [self.flat[o:o + n_out * n_in].reshape(shape) for o in offsets]
        depth, self.cols = (n_out, n_in) if input_grad else (n_in, n_out)
        self.rows = sum(counts) + behind
        self.x, self.xv = device_rows(draw(self.rows, depth), True, x_pad, offset)
        self.wide = torch.full((self.rows + 2, self.cols + y_pad), 7.5, device="cuda",
                               dtype=torch.bfloat16 if bf16 else torch.float32)
        self.y = self.wide[1:self.rows + 1, :self.cols]
        query = zr.zr_linear_input_grad_workspace if input_grad else zr.zr_linear_forward_workspace
        nbytes = query(self.plan, self.params, counts, n_out, n_in, in_major)
        self.ws = workspace(nbytes) if nbytes else None

    def call(self, stream=None):
        fn = zr.zr_linear_input_grad if self.input_grad else zr.zr_linear_forward
        fn(self.plan, self.params, self.counts, self.parts, self.x, self.y, in_major=self.in_major,
           workspace=self.ws, stream=stream)

    def check(self, exact=False):
        torch.cuda.synchronize()
        wide = self.wide.double().cpu().numpy()
        at = sum(self.counts)
        assert (wide[0] == 7.5).all() and (wide[1 + at:] == 7.5).all() and (wide[:, self.cols:] == 7.5).all()
        at = 1
        for w, c in zip(self.weights, self.counts):
            x = self.xv[at - 1:at - 1 + c]
            m = w if self.input_grad != self.in_major else w.T
            want, size = x @ m, np.abs(x) @ np.abs(m)
            got = wide[at:at + c, :self.cols]
            tol = 0.0 if exact else (x.shape[1] * 2 * U * size + (2.0 ** -8 if self.bf16 else 0) * np.abs(want)) * 1.01
            bad = np.abs(got - want) > tol
            assert not bad.any(), (c, int(bad.sum()), np.argwhere(bad)[0], got[bad][0], want[bad][0])
            at += c


BOTH = [(i, m) for i in (False, True) for m in (False, True)]
SHAPES = [
    # one value; less than a tile of anything; more, odd
    (1, 1, [1], 1, 0), (3, 5, [2, 0, 7], 2, 1), (130, 70, [33, 1], 3, 5), (257, 129, [65, 300], 2, 0),
    # rows on 16 bytes: whole tiles, and ragged ones
    (256, 128, [256], 1, 0), (512, 192, [257, 0, 64, 511], 2, 8), (264, 328, [100, 31], 3, 16),
    # few rows, sums in pieces
    (2304, 768, [1], 1, 0), (200, 4096, [3, 17, 32, 64], 8, 0), (96, 8200, [1, 2], 5, 3),
    # many partitions in a weight, and in a step of it
    (300, 100, [70, 5], 64, 0), (24, 40, [9], 64, 0), (1000, 520, [129], 7, 8)]


@pytest.mark.parametrize("input_grad,in_major", BOTH)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}-{len(s[2])}-{s[3]}")
def test_products(shape, input_grad, in_major):
    n_out, n_in, counts, world, lead = shape
    even = n_out % 8 == 0 and n_in % 8 == 0 and lead % 8 == 0
    for k, kw in enumerate((dict(align=8 if even else 1), dict(bf16=False, x_pad=8 if even else 3, y_pad=3, behind=5,
                                                              align=8 if even else 1),
                            dict(offset=1, part_offset=3, x_pad=1))):
        c = Case(k, n_out, n_in, counts, input_grad, in_major, world, lead, **kw)
        c.call()
        c.check()


@pytest.mark.parametrize("input_grad,in_major", BOTH)
def test_whole_numbers(input_grad, in_major):
    """Every sum is exact, whatever the tiles and pieces."""
    for seed, (n_out, n_in, counts, kw) in enumerate((
            (768, 512, [700, 3, 0, 1030], dict(align=8, world=2)), (770, 515, [700, 3, 0, 1030], dict(world=3)),
            (512, 4096, [5, 33, 64], dict(align=8)), (2048, 640, [1], dict()))):
        c = Case(seed, n_out, n_in, counts, input_grad, in_major, bf16=False, whole=True, **kw)
        c.call()
        c.check(exact=True)


# (rows, columns, depth) that every shape of tiles is the choice for, with its sums
# whole and in pieces, on 16 bytes and off them
TILES = [(30, 256, 64), (9, 128, 9600), (300, 1024, 256), (42, 32, 2048), (4118, 928, 64), (3609, 32, 9520),
         (2886, 4240, 144), (149, 11520, 4096)]


@pytest.mark.parametrize("off", (0, 1))
@pytest.mark.parametrize("columns", (False, True))
@pytest.mark.parametrize("tiles", TILES, ids=lambda t: "x".join(map(str, t)))
def test_every_shape_of_tiles(tiles, columns, off):
    rows, cols, depth = tiles[0], tiles[1] + off, tiles[2] + off
    n_out, n_in = (depth, cols) if columns else (cols, depth)
    c = Case(5, n_out, n_in, [rows], columns, bf16=False, whole=True, world=2, align=1 if off else 8)
    c.call()
    c.check(exact=True)


@pytest.mark.parametrize("counts", ([3], [70], [900]))
def test_rows_on_16_bytes_with_a_ragged_end(counts):
    """What stands behind a row's last element is not multiplied."""
    for k, (n_out, n_in) in enumerate(((203, 128), (1001, 256))):
        c = Case(k, n_out, n_in, counts, True, align=8, bf16=False, whole=True)
        wide = torch.full((c.rows, (n_out + 7) // 8 * 8), float("nan"), device="cuda", dtype=torch.bfloat16)
        wide[:, :n_out] = c.x
        c.x = wide[:, :n_out]
        c.call()
        c.check(exact=True)


def test_many_groups_and_repeated_weights():
    rng = np.random.default_rng(0)
    for n, most in ((300, 5), (140, 90)):
        counts = [int(v) for v in rng.integers(0, most, n)]
        for input_grad in (False, True):
            c = Case(1, 48, 64, counts, input_grad, align=8, params=[int(v) for v in rng.integers(0, 6, n)])
            c.call()
            c.check()


def test_non_finite_values_stay_in_their_rows_and_weights():
    for n_out, n_in, counts in ((264, 136, [70, 40]), (264, 136, [3, 9]), (131, 77, [70, 40]), (131, 77, [3, 9])):
        for input_grad, in_major in BOTH:
            c = Case(2, n_out, n_in, counts, input_grad, in_major, behind=4, bf16=False, align=8)
            c.x[1, 5] = float("nan")
            c.x[counts[0], 3] = float("inf")
            c.x[-4:] = float("nan")
            c.call()
            y = c.y[:sum(counts)].cpu().numpy()
            good = np.ones(len(y), bool)
            good[[1, counts[0]]] = False
            assert np.isnan(y[1]).all() and not np.isfinite(y[counts[0]]).any()
            c.xv[[1, counts[0]]] = 0
            c.y[1] = 0
            c.y[counts[0]] = 0
            assert np.isfinite(y[good]).all()
            c.check()
            # a weight's NaN touches its column and its group only
            c = Case(2, n_out, n_in, counts, input_grad, in_major, bf16=False, align=8)
            flat = c.parts[0]
            o = zr.zr_plan_param_offset(c.plan, c.params[1])
            flat[o] = float("nan")
            c.call()
            y = c.y.cpu().numpy()
            assert np.isfinite(y[:counts[0]]).all() and np.isnan(y[counts[0]:, 0]).all()
            assert np.isfinite(y[counts[0]:, 1:]).all()


def test_bits_do_not_depend_on_where_things_lie():
    for n_out, n_in, counts in ((512, 264, [300, 65]), (512, 4104, [3, 64])):
        for input_grad, in_major in BOTH:
            got = []
            for kw in (dict(), dict(offset=1), dict(part_offset=1), dict(x_pad=3, y_pad=1), dict(world=3)):
                c = Case(3, n_out, n_in, counts, input_grad, in_major, align=8, **kw)
                c.call()
                torch.cuda.synchronize()
                got.append(c.y.clone())
            assert all(torch.equal(got[0], g) for g in got[1:])


def test_two_streams_and_graphs():
    cases = [Case(4, 512, 1024, [5, 20], False, align=8), Case(5, 512, 1024, [5, 20], True, align=8),
             Case(6, 776, 520, [600, 0, 70], False, True, align=8), Case(7, 775, 521, [600, 0, 70], True)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for s, c in zip(streams, cases):
            c.call(stream=s)
    for c in cases:
        c.check()
        eager = c.y.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        for _ in range(3):
            c.wide.fill_(7.5)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(eager, c.y)
            torch.randn(1000, device="cuda").sum().item()
        c.check()


def test_two_graphs_share_a_workspace():
    """Sums in pieces: nothing in the workspace outlives a call."""
    cases = [Case(8, 264, 8192, [3], False, align=8), Case(9, 8192, 256, [70], True, align=8),
             Case(10, 131, 9001, [40], False)]
    ws = workspace(max(c.ws.numel() for c in cases))
    graphs = []
    for c in cases:
        c.ws = ws
        c.call()
        c.check()
        graphs.append((torch.cuda.CUDAGraph(), c.y.clone()))
        with torch.cuda.graph(graphs[-1][0]):
            c.call()
    for _ in range(3):
        for (g, eager), c in zip(graphs, cases):
            c.wide.fill_(7.5)
            g.replay()
            c.call()
            assert torch.equal(eager, c.y)
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """A weight behind 2^32 bytes of its partition, and outputs of more."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    lead, o, i = (1 << 31) + 8, 4096, 64
    plan = zr.zr_plan_buckets([lead, o * i], [0, 0], [(1, 1)], 1 << 40)
    flat = torch.empty(lead + o * i, dtype=torch.bfloat16, device="cuda")
    w = flat[lead:].view(o, i)
    w.normal_(generator=gen)
    rows = (1 << 31) // o + 300
    x = torch.empty(rows, i, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    y = torch.empty(rows, o, dtype=torch.bfloat16, device="cuda")
    zr.zr_linear_forward(plan, [1], [rows], [flat], x, y)
    size = lambda a, b: a.double().abs() @ b.double().abs()  # noqa: E731
    for at in (0, rows // 2, rows - 300):
        want = x[at:at + 300].double() @ w.double().t()
        tol = i * 2 * U * size(x[at:at + 300], w.t()) + 2.0 ** -8 * want.abs()
        assert ((y[at:at + 300].double() - want).abs() <= 1.01 * tol).all()
    dx = torch.empty(rows, i, device="cuda")
    zr.zr_linear_input_grad(plan, [1], [rows], [flat], y, dx)
    for at in (0, rows // 2, rows - 300):
        want = y[at:at + 300].double() @ w.double()
        assert ((dx[at:at + 300].double() - want).abs() <= 1.01 * o * 2 * U * size(y[at:at + 300], w)).all()


def test_refusals():
    plan = zr.zr_plan_buckets([8 * 16, 8 * 16], [0, 0], [(2, 1)], 1000)
    P = zr.zr_plan_group_info(plan, 0)[2]
    parts = [torch.zeros(P, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x, y = torch.zeros(5, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 8, device="cuda")

    def refused(match, *args, call=zr.zr_linear_forward, **kw):
        with pytest.raises(zr.ZrError, match=match):
            call(plan, *args, **kw)
    refused("x must be", [0, 1], [2, 3], parts, x.float(), y)
    refused("y must be", [0, 1], [2, 3], parts, x, y.half())
    refused("y has shape", [0, 1], [2, 3], parts, x, y[:4])
    refused("contiguous rows", [0, 1], [2, 3], parts, x.t(), y)
    refused("parts has 1", [0, 1], [2, 3], parts[:1], x, y)
    refused(r"parts\[1\] holds", [0, 1], [2, 3], [parts[0], parts[1][1:]], x, y)
    refused(r"parts\[0\] must be", [0, 1], [2, 3], [parts[0].float(), parts[1]], x, y)
    refused("partition 1 is null", [0, 1], [2, 3], [parts[0], None], x, y)
    refused("counts has", [0, 1], [2], parts, x, y)
    refused("add up", [0, 1], [2, 4], parts, x, y)
    refused("n_out \\* n_in", [0, 1], [2, 3], parts, x, y[:, :7])
    refused("param id", [0, 2], [2, 3], parts, x, y)
    refused("dy must be", [0, 1], [2, 3], parts, y, x, call=zr.zr_linear_input_grad)
    refused("on|device", [0, 1], [2, 3], [parts[0], parts[1].cpu()], x, y)
    assert y.abs().max() == 0

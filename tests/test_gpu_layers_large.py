"""The layer operators where offsets pass 32 bits, on whole numbers (exact sums
and values); and several calls on the GPU at once."""

import pytest

from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")

TABLE = (1 << 20) + 3, 4100         # 4.3e9 elements


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def test_lookup_in_a_table_of_more_than_2_32_elements():
    vocab, dim = TABLE
    plan = zr.zr_plan_buckets([vocab * dim], [0], [(1, 1)], 1 << 50)
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab, (1 << 32) // dim, (1 << 31) // dim, vocab - 2], device="cuda")
    some = torch.randint(-100, 101, (6, dim), device="cuda").bfloat16()
    some[2] = 0
    for i in (0, 1, 3, 4, 5):
        table[ids[i]] = some[i]
    out = torch.empty(6, dim, dtype=torch.bfloat16, device="cuda")
    zr.zr_embedding_lookup(plan, 0, dim, [table.view(-1)], ids, out)
    assert torch.equal(out, some)


@pytest.mark.parametrize("few", [True, False])
def test_embedding_gradient_of_more_than_2_32_elements(few):
    """Zeros before the sums (few tokens of many rows) and beside them."""
    vocab, dim = TABLE if few else (5000, 900001)
    plan = zr.zr_plan_buckets([7, vocab * dim], [0, 0], [(1, 1)], 1 << 50)
    n = 300 if few else 1400
    ids = torch.randint(0, vocab, (n,), device="cuda")
    ids[::3] = vocab - 1 - ids[::3] % 3
    dy = torch.randint(-4, 5, (n, dim), device="cuda", dtype=torch.int8).bfloat16()
    length = 7 + vocab * dim
    grad = torch.full((length,), 3.0, device="cuda")
    size = zr.zr_ipg_embedding_workspace(plan, 1, dim, n, 0, length)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    zr.zr_ipg_accumulate_embedding_first(plan, 1, dim, ids, dy, grad, ws)
    zr.zr_ipg_accumulate_embedding(plan, 1, dim, ids, dy, grad, ws, scale=2.0)
    assert (grad[:7] == 3.0).all()
    got = grad[7:].view(vocab, dim)
    for row in ids.unique().tolist():
        want = dy[ids == row].double().sum(0).float()
        assert torch.equal(got[row], 3 * want), row
        got[row] = 0
    assert sum(int(torch.count_nonzero(x)) for x in got.split(max(1, vocab // 16))) == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_checkpoint_of_more_than_2_32_values(bf16):
    rows, cols = 131101, 32800
    dtype = torch.bfloat16 if bf16 else torch.float32
    codes, scales = zr.act_empty(rows, cols)
    row = torch.randint(-15, 16, (cols,), device="cuda").to(dtype)
    x = row.repeat(rows, 1)
    x[-1] *= 2
    x[rows // 2] = 0
    zr.zr_act_quantize(x, codes, scales)
    out = torch.full((rows, cols), 7.5, dtype=dtype, device="cuda")
    zr.zr_act_dequantize(codes, scales, out)
    for a, b in zip(out.split(8192), x.split(8192)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("in_major", [False, True])
@pytest.mark.parametrize("n_out,n_in,tokens,lead", [(4096, 260, 530001, 0), (4100, 260, 530001, 1),
                                                    (264, 8192, 530003, 0)])
def test_linear_gradient_of_operands_of_more_than_2_32_bytes(n_out, n_in, tokens, lead, in_major):
    """dY's rows on 16 bytes and off them, and X's codes."""
    plan = zr.zr_plan_buckets([n_out * n_in], [0], [(1, 1)], 1 << 40)
    flat = torch.zeros(tokens * n_out + lead, dtype=torch.bfloat16, device="cuda")
    dy = flat[lead:].view(tokens, n_out)
    codes, scales = zr.act_empty(tokens, n_in)
    want = torch.zeros(n_in if in_major else n_out, n_out if in_major else n_in, device="cuda",
                       dtype=torch.float64)
    for t in range(0, tokens, 1 << 16):     # +-1 and 0: sums below 2^24
        m = min(1 << 16, tokens - t)
        d = torch.randint(-1, 2, (m, n_out), device="cuda", dtype=torch.int8).bfloat16()
        x = torch.randint(-1, 2, (m, n_in), device="cuda", dtype=torch.int8).float()
        dy[t:t + m] = d
        zr.zr_act_quantize(x, codes[t:t + m], scales[t:t + m])
        a, b = (x, d.float()) if in_major else (d.float(), x)
        want += (a.t().contiguous() @ b).double()
    items = [(0, dy, codes, scales, in_major)]
    grad = torch.empty(n_out * n_in, device="cuda")
    ws = torch.empty(zr.zr_ipg_linear_workspace(plan, items, 0, n_out * n_in), dtype=torch.uint8, device="cuda")
    zr.zr_ipg_accumulate_linear_first(plan, items, grad, ws)
    assert torch.equal(grad.double().view(want.shape), want) and want.abs().max() > 100


def test_calls_on_two_streams_at_once():
    """A workspace each: both give what they give alone, call after call."""
    torch.manual_seed(0)
    plan = zr.zr_plan_buckets([3000 * 260, 700 * 260], [0, 0], [(1, 1)], 1 << 40)
    n, length = 4000, 3700 * 260
    work = []
    for _ in range(2):
        ids = torch.randint(-5, 3000, (n,), device="cuda")
        dx = torch.randn(n, 260, device="cuda").bfloat16()
        codes, scales = zr.act_empty(n, 260)
        zr.zr_act_quantize(torch.randn(n, 260, device="cuda"), codes, scales)
        items = [(1, torch.randn(n, 700, device="cuda").bfloat16(), codes, scales)]
        ws = torch.empty(max(zr.zr_ipg_linear_workspace(plan, items, 0, length),
                             zr.zr_ipg_embedding_workspace(plan, 0, 260, n, 0, length)),
                         dtype=torch.uint8, device="cuda")
        work.append((ids, dx, items, ws))

    def step(k, grad, stream=None):
        ids, dx, items, ws = work[k]
        zr.zr_ipg_accumulate_embedding_first(plan, 0, 260, ids, dx, grad, ws, stream=stream)
        zr.zr_ipg_accumulate_linear_first(plan, items, grad, ws, stream=stream)
        zr.zr_ipg_accumulate_linear(plan, items, grad, ws, stream=stream)
        zr.zr_ipg_accumulate_embedding(plan, 0, 260, ids, dx, grad, ws, stream=stream)

    want = [torch.empty(length, device="cuda") for _ in range(2)]
    for k in range(2):
        step(k, want[k])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty(length, device="cuda") for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for r in range(8):
        for k in range(2):
            step(k, got[k][r], streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for r in range(8):
            assert torch.equal(got[k][r], want[k])

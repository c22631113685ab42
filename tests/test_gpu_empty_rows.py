"""Matrices without rows whose columns lie apart, on the GPU: the older layer
calls refuse them as they do any such matrix, the products and losses return."""

import pytest

from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")


def _apart(cols, dtype=torch.bfloat16):
    t = torch.empty(0, 2 * cols, dtype=dtype, device="cuda")[:, ::2]
    assert t.stride(1) == 2
    return t


def test_older_calls_refuse_them():
    plan = zr.zr_plan_buckets([8 * 16], [0], [(1, 1)], 1000)
    P = zr.zr_plan_group_info(plan, 0)[2]
    part, ids = torch.zeros(P, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    for call in (lambda: zr.zr_act_quantize(_apart(16), *zr.act_empty(0, 16)),
                 lambda: zr.zr_act_dequantize(*zr.act_empty(0, 16), _apart(16)),
                 lambda: zr.zr_embedding_lookup(plan, 0, 16, [part], ids, _apart(16)),
                 lambda: zr.zr_ipg_linear_workspace(plan, [(0, _apart(8), *zr.act_empty(0, 16))], 0, P)):
        with pytest.raises(zr.ZrError, match="contiguous rows"):
            call()


def test_products_and_losses_return():
    plan = zr.zr_plan_buckets([8 * 16], [0], [(1, 1)], 1000)
    P = zr.zr_plan_group_info(plan, 0)[2]
    parts = [torch.zeros(P, dtype=torch.bfloat16, device="cuda")]
    zr.zr_linear_forward(plan, [0], [0], parts, _apart(16), _apart(8))
    zr.zr_linear_input_grad(plan, [0], [0], parts, _apart(8), _apart(16))
    none, tokens = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    zr.zr_distill_loss(_apart(9), _apart(3, torch.int64), _apart(3, torch.float32), None, none, _apart(9))
    zr.zr_policy_loss(_apart(9), tokens, none, None, none, None, none, none, _apart(9))
    torch.cuda.synchronize()

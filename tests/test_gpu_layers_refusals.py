"""What the layer calls' binding refuses of device tensors: nothing is enqueued."""

import pytest

from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")


def _refused(match, call, *args, **kwargs):
    with pytest.raises(zr.ZrError, match=match) as e:
        call(*args, **kwargs)
    assert e.value.status == zr.ZR_ERR_INVALID


def test_rows_that_are_not_contiguous_and_wrong_shapes():
    x = torch.zeros(8, 64, device="cuda")
    codes, scales = zr.act_empty(64, 8)
    _refused("contiguous rows", zr.zr_act_quantize, x.t(), codes, scales)
    codes, scales = zr.act_empty(8, 64)
    _refused("contiguous rows", zr.zr_act_quantize, x[:1].expand(8, 64), codes, scales)
    _refused("contiguous rows", zr.zr_act_quantize, x[:, ::2], *zr.act_empty(8, 32))
    _refused("contiguous rows", zr.zr_act_dequantize, codes, scales, x[:1].expand(8, 64))
    _refused("have shapes", zr.zr_act_quantize, x[:7], codes, scales)
    _refused("codes must be", zr.zr_act_quantize, x, codes.view(torch.uint8), scales)
    _refused("codes must be contiguous", zr.zr_act_quantize, x[:, :32],
             torch.empty(8, 64, dtype=torch.float8_e4m3fn, device="cuda")[:, :32], scales[:, :1])
    _refused("scales must be a device", zr.zr_act_quantize, x, codes, scales.cpu())


def test_lookup_and_gradients():
    plan = zr.zr_plan_buckets([10 * 8, 4 * 8], [0, 0], [(2, 1)], 1000)
    P = zr.zr_plan_group_info(plan, 0)[2]
    parts = [torch.zeros(P, device="cuda") for _ in range(2)]
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    out, grad = torch.zeros(3, 8, device="cuda"), torch.zeros(2 * P, device="cuda")
    _refused("parts has 1 entries", zr.zr_embedding_lookup, plan, 0, 8, parts[:1], ids, out)
    _refused(r"parts\[1\] holds", zr.zr_embedding_lookup, plan, 0, 8, [parts[0], parts[1][1:]], ids, out)
    _refused(r"parts\[0\] must be torch.float32", zr.zr_embedding_lookup, plan, 0, 8,
             [parts[0].bfloat16(), parts[1]], ids, out)
    _refused("out has shape", zr.zr_embedding_lookup, plan, 0, 8, parts, ids, out[:2])
    _refused("tokens must be contiguous", zr.zr_embedding_lookup, plan, 0, 8, parts, ids.repeat(2)[::2], out)
    _refused("dim", zr.zr_embedding_lookup, plan, 0, 9, parts, ids, torch.zeros(3, 9, device="cuda"))
    ws = torch.zeros(zr.zr_ipg_embedding_workspace(plan, 0, 8, 3, 0, 2 * P), dtype=torch.uint8, device="cuda")
    for call in (zr.zr_ipg_accumulate_embedding, zr.zr_ipg_accumulate_embedding_first):
        _refused("workspace is null", call, plan, 0, 8, ids, out, grad, ws[:-16])
        _refused("dy has shape", call, plan, 0, 8, ids, out[:, :7], grad, ws)
        _refused("main_grad holds", call, plan, 0, 8, ids, out, grad, ws, window_len=2 * P + 1)
        _refused("window runs past", call, plan, 0, 8, ids, out, grad, ws, window_base=1)
    dy = torch.zeros(4000, 4, dtype=torch.bfloat16, device="cuda")
    item = (1, dy, *zr.act_empty(4000, 8))
    need = zr.zr_ipg_linear_workspace(plan, [item], 0, 2 * P)
    assert need > 0
    for call in (zr.zr_ipg_accumulate_linear, zr.zr_ipg_accumulate_linear_first):
        _refused("workspace is null", call, plan, [item], grad, None)
        _refused("workspace is null", call, plan, [item], grad,
                 torch.zeros(need - 16, dtype=torch.uint8, device="cuda"))
        _refused("dy must be one of", call, plan, [(1, dy.float(), *item[2:])], grad, None)
        _refused("have shapes", call, plan, [(1, dy[:-1], *item[2:])], grad, None)
        _refused("twice", call, plan, [item, item], grad, None)
    assert grad.abs().max() == 0 and out.abs().max() == 0

"""Arguments that do not fit the C call's types are refused, not cut down, and
what older calls refuse stays refused.  Made without a GPU."""

import pytest

from tests._lib import load

zr = load()
torch = pytest.importorskip("torch")


def _plan():
    return zr.zr_plan_buckets([48, 48], [0, 0], [(2, 1)], 1000)


@pytest.mark.parametrize("query", [zr.zr_linear_forward_workspace, zr.zr_linear_input_grad_workspace])
@pytest.mark.parametrize("params,counts,words", [
    ([2 ** 64], [3], "params"), ([-2 ** 63 - 1], [3], "params"), ([0, 2 ** 64 + 1], [3, 4], "params"),
    ([0], [2 ** 64 + 3], "counts"), ([0, 1], [3, 2 ** 63], "counts"), ([0], [-2 ** 64 + 3], "counts"),
    ([0.0], [3], "integers"), ([0], [3.0], "integers"), ([0], ["3"], "integers"), ([None], [3], "integers"),
])
def test_lists_past_64_bits(query, params, counts, words):
    with pytest.raises(zr.ZrError, match=words):
        query(_plan(), params, counts, 8, 6)


def test_lists_that_fit():
    for query in (zr.zr_linear_forward_workspace, zr.zr_linear_input_grad_workspace):
        for params, counts in (([0, 1], [3, 4]), ((1,), (0,)), ([], []), ([0, 1], range(2))):
            assert query(_plan(), params, counts, 8, 6) >= 0
        # the C call's own check
        with pytest.raises(zr.ZrError, match="param id"):
            query(_plan(), [2 ** 63 - 1], [3], 8, 6)


def test_empty_rows_with_strided_columns():
    """Refused by the older layer calls; the products and losses take them, as
    there is nothing to read."""
    t = torch.empty(0, 6)[:, ::2]
    assert t.stride(1) == 2
    with pytest.raises(zr.ZrError, match="contiguous rows"):
        zr._rows(t, "x", t.get_device())
    assert zr._rows(t, "x", t.get_device(), empty=True) == (t.data_ptr(), 6)
    with pytest.raises(zr.ZrError, match="contiguous rows"):
        zr._rows(torch.empty(2, 6)[:, ::2], "x", -1, empty=True)


@pytest.mark.parametrize("kl", [3.5e38, -1e300])
def test_kl_that_fp32_does_not_hold(kl):
    """The kernels take it in fp32: infinite there, times a term of 0."""
    one, A = (3, 10, 10), 0x10000
    status = zr._lib.zr_policy_loss(A, zr.ZR_BF16, *one, A, zr.ZR_I64, A, A, A, A, 0.2, 0.2, kl, 1.0, A, A, A, 10,
                                    None, 0, None)
    assert status == zr.ZR_ERR_INVALID and "kl must" in zr.zr_last_error()

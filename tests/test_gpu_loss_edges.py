"""The losses at the ends of what their arguments may hold, on the GPU: rows of
chosen values in the forms that take a row to a workgroup and that cut it into
pieces.  Where values are compared, tolerances are those of test_gpu_losses.py."""

import numpy as np
import pytest

from oracle.losses import softmax_oracle
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._layers import U  # noqa: E402
from tests.test_gpu_losses import Case  # noqa: E402

# whole rows, rows in pieces, and several rows to a workgroup
FORMS = [(9, 300), (9, 40000), (160, 1500), (600, 66000)]


def _put(c, **values):
    """Replaces the first rows' numbers of a case: weight, old, ref, advantage."""
    for name, v in values.items():
        host, dev = dict(weight=(c.w, c.weight), old=(c.old, c.per[0]), ref=(c.ref, c.per[1]),
                         advantage=(c.adv, c.per[2]))[name]
        host[:len(v)] = v
        dev.copy_(torch.from_numpy(host))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_rows_of_weight_0(rows, vocab, bf16, in_place):
    """Zeros, whatever the row holds; its log-probability is still given."""
    def values(z):
        z[0, 5], z[1, 5], z[2, 5] = np.nan, np.inf, -np.inf
        z[3, :] = -np.inf
    for top in (0, 3):
        c = Case(np.random.default_rng(3), rows, vocab, bf16, top=top, kl=0.3, values=values, in_place=in_place)
        c.ids[:6] = [[7, 8, 9]] * 6 if top else 7
        c.ids_dev.copy_(torch.from_numpy(c.ids))
        _put(c, weight=[0.0] * 5, advantage=[1.0, 1.0, 1.0, 1.0, np.nan], ref=[-3.0, -3.0, -3.0, -3.0, np.nan])
        c.call()
        c.check([2, 5, 6, 7, rows - 1])
        bits = c.dlogits[:5].contiguous().view(torch.int16 if bf16 else torch.int32)
        assert (bits == 0).all() and (c.loss[:5] == 0).all()
        if not top:
            logp = c.logp[:5].cpu().numpy()
            assert np.isnan(logp[:2]).all() and np.isfinite(logp[[2, 4]]).all() and logp[3] == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_references_far_from_the_policy(rows, vocab, bf16):
    far = [-100.0, -1e6, -1.7e7, -3e7, -1e8, -1e9, 5.0, -np.inf]
    c = Case(np.random.default_rng(4), rows, vocab, bf16, kl=0.5)
    c.ids[:8] = 7
    c.ids_dev.copy_(torch.from_numpy(c.ids))
    _put(c, ref=far, advantage=[0.0] * 8)
    c.call()
    c.check(list(range(7)) + [rows - 1])
    # no reference at all: an infinite loss, whose slope is kl
    got = c.dlogits[7].double().cpu().numpy()
    q = torch.softmax(torch.from_numpy(c.z[7]), 0).numpy()
    q[7] -= 1
    assert c.loss[7] == np.inf
    # c.check's bound for a multiple of 0.5 w
    part = U * (3 * np.log(vocab) + vocab / 256 + 210)
    want = -0.5 * c.w[7] * q
    tol = 1.01 * (0.5 * c.w[7] * (np.abs(q) * (part + 300 * U) + 11 * U) + (2.0 ** -8 if bf16 else U) * np.abs(want))
    assert (np.abs(got - want) <= tol + 2.0 ** -126).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_ratios_that_fp32_does_not_hold(rows, vocab, bf16):
    """Large ones by their own formula, infinite ones, and any of them with an
    advantage of 0."""
    c = Case(np.random.default_rng(5), rows, vocab, bf16, weighted=False)
    lp = [c.z[i] - np.log(np.exp(c.z[i]).sum()) for i in range(9)]
    old = np.float32([lp[i][7] - x for i, x in enumerate((60, 100, 500, 100, 1e9, 100, 1e9, 1e9, -1e9))])
    adv = np.float32([-1e-20, -1e-20, -1e-20, -1e-30, -1e-30, 0.0, 0.0, 1.0, -1.0])
    old[6] = -np.inf
    c.ids[:9] = 7
    c.ids_dev.copy_(torch.from_numpy(c.ids))
    _put(c, old=old, advantage=adv)
    c.call()
    c.check([0, 3, 5, rows - 1])
    loss, g = c.loss.cpu().numpy(), c.dlogits.float().cpu().numpy()
    want = [1e-20 * np.exp(lp[i][7] - float(old[i])) for i in (0, 1)]
    assert np.isclose(loss[0], want[0], rtol=1e-4) and np.isclose(loss[1], want[1], rtol=1e-4)
    assert loss[2] == np.inf and loss[4] == np.inf and (loss[5:7] == 0).all()
    # clipped on either side: the border's loss, and no gradient
    assert np.isclose(loss[7:9], [-1.28, 0.8], rtol=1e-6).all()
    assert (g[5:9] == 0).all() and g[2, 7] == np.inf


@pytest.mark.parametrize("tau", [1.0, 1e-8, 1e8])
@pytest.mark.parametrize("top", [0, 2])
@pytest.mark.parametrize("vocab", [300, 9001])
def test_rows_far_from_0(vocab, top, tau):
    """Around 10^8 binary orders from 0, steps of fp32 apart."""
    at, rows = 1e8 * np.log(2) * tau, 116

    def values(z):
        for i in range(rows):
            first = (-1) ** i * at * (1 + (i // 4 - 8) * 2.0 ** -23)
            z[i] = first - at * 2.0 ** -23 * (np.arange(vocab) % 5)
            if i % 4 > 1:
                z[i, 1::7] = 0.5
    c = Case(np.random.default_rng(6), rows, vocab, False, top=top, tau=tau, values=values)
    if not top:   # the row's highest: fp32 holds no ratio to one that is 10^8 orders below
        c.ids = c.z.argmax(1)
        c.ids_dev.copy_(torch.from_numpy(c.ids))
        _put(c, old=np.float32([0.1 + softmax_oracle(z, tau)[1].max() for z in c.z]))
    c.call()
    c.check(range(rows))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_multiples_that_fp32_does_not_hold(rows, vocab, bf16, in_place):
    """Each column's gradient is its own: masked ones 0, others finite while fp32
    holds them."""
    def values(z):
        z[:9, 3::11] = -np.inf
        z[:9, 4::11] = -150.0
    c = Case(np.random.default_rng(7), rows, vocab, bf16, weighted=False, values=values, in_place=in_place)
    c.ids[:9] = 9
    c.ids_dev.copy_(torch.from_numpy(c.ids))
    lp = np.array([softmax_oracle(c.z[i], 1.0)[1][9] for i in range(9)])
    old = (lp - [60, 70, 80, 86, 89, 91, 95, 150, 400]).astype(np.float32)
    _put(c, old=old, advantage=np.float32([-0.5] * 9))
    c.call()
    c.check([rows - 1] if rows > 9 else [])
    got = c.dlogits[:9].double().cpu().numpy()
    part = U * (3 * np.log(vocab) + vocab / 256 + 210)
    for i in range(9):
        q = softmax_oracle(c.z[i], 1.0)[0]
        q[9] -= 1
        # the ratio is off by what log q is and 8 U, q by its part and 3 U an order
        want = -0.5 * np.exp(lp[i] - float(old[i])) * q
        rel = 2 * part + 3 * U * abs(lp[i]) + 3 * U * 160 + 16 * U + (2.0 ** -8 if bf16 else U)
        most = float(torch.finfo(c.dlogits.dtype).max)
        sure = np.abs(np.abs(want) / most - 1) > 2 * rel
        assert (got[i, 3::11] == 0).all()
        held = sure & (np.abs(want) < most)
        tol = 1.01 * rel * np.abs(want[held]) + 2.0 ** -126 * (1 + min(np.exp(lp[i] - float(old[i])), 1e30))
        assert (np.abs(got[i][held] - want[held]) <= tol).all(), i
        past = sure & ~held
        assert (got[i][past] == np.sign(want[past]) * np.inf).all(), i
    assert held.any() and past.any()

"""Losses over more than 2^32 bytes of logits, every row of them: log-probabilities
against 64 bits, and each gradient's row sums."""

import numpy as np
import pytest

from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._layers import U, workspace  # noqa: E402

ROWS, VOCAB, STEP = 17000, 128256, 500


def test_every_row_past_32_bits():
    gen = torch.Generator(device="cuda").manual_seed(2)
    z = torch.empty(ROWS, VOCAB, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    tokens = torch.randint(VOCAB, (ROWS,), generator=gen, device="cuda")
    # each row's own weight, so that no row's gradient passes for another's
    weight = 0.5 + torch.rand(ROWS, generator=gen, device="cuda")
    old = torch.full((ROWS,), -12.0, device="cuda")
    loss, logp = (torch.full((ROWS,), float("nan"), device="cuda") for _ in range(2))
    g = torch.full_like(z, float("nan"))
    zr.zr_policy_loss(z, tokens, old, None, torch.full_like(old, -1.0), weight, loss, logp, g,
                      workspace=workspace(zr.zr_loss_workspace(ROWS, VOCAB, 1, z.dtype)))
    # as in test_gpu_losses.py: what a row's sum adds to q, of it, and to log q
    part = U * (3 * np.log(VOCAB) + VOCAB / 256 + 210)
    left_out = 0
    for i in range(0, ROWS, STEP):
        here = slice(i, i + STEP)
        x = z[here].double()
        lp = x.gather(1, tokens[here, None])[:, 0] - x.logsumexp(1)
        off = part + 4 * U * lp.abs()
        assert ((logp[here].double() - lp).abs() <= off).all(), i
        # advantage -1: the loss is the ratio, or the border 0.8
        r = (lp - old[here].double()).exp()
        w = weight[here].double()
        inside = r > 0.8
        # a ratio within its error of the border may fall on either side: the few
        # such rows (1e-4 of them) are left out of what follows
        sure = (r / 0.8 - 1).abs() > 2 * off
        left_out += int((~sure).sum())
        want = w * torch.where(inside, r, 0.8)
        assert ((loss[here].double() - want).abs() <= 1.01 * (off + 10 * U) * want)[sure].all(), i
        # w r (1[v = a] - q): the token's element is the others' sum, a row's sizes
        # add up to 2 w r (1 - q_a); each is off by its type's half step and by twice
        # the row's part
        f = g[here].double()
        size = torch.where(inside, 2 * w * r * (1 - lp.exp()), 0.0)
        tol = 1.01 * (2.0 ** -8 + 2 * off + 10 * U) * size
        assert ((f.abs().sum(1) - size).abs() <= tol)[sure].all(), i
        assert (f.sum(1).abs() <= tol)[sure].all(), i
        at = f.gather(1, tokens[here, None])[:, 0]
        assert ((at - size / 2).abs() <= tol)[sure].all(), i
    assert inside.any() and not inside.all() and left_out < 20

"""The losses' oracle: values by hand, gradients against torch's autograd of
the definitions and against central differences."""

import numpy as np
import pytest

from oracle.losses import distill_oracle, policy_oracle, softmax_oracle

torch = pytest.importorskip("torch")


def test_softmax_by_hand():
    q, log_q = softmax_oracle(np.array([0.0, np.log(3.0), -np.inf]), 1.0)
    assert np.allclose(q, [0.25, 0.75, 0.0], atol=1e-15) and log_q[2] == -np.inf
    q, _ = softmax_oracle(np.array([0.0, np.log(3.0)]), 0.5)
    assert np.allclose(q, [0.1, 0.9], atol=1e-15)


def test_distill_by_hand():
    # the teacher's whole row: the loss is KL(p || q); equal rows give 0
    z = np.array([1.0, 2.0, 0.5])
    loss, coef, q, target, _ = distill_oracle(z, [0, 1, 2], z, 2.0, 1.5)
    assert abs(loss) < 1e-15 and np.allclose(q, target, atol=1e-15) and coef == 3.0
    # one entry: the cross-entropy
    loss, _, q, target, _ = distill_oracle(z, [1, -1, 3], z, 1.0, 1.0)
    assert np.isclose(loss, -np.log(q[1]), atol=1e-15) and list(target) == [0, 1, 0]
    # an entry twice
    _, _, _, target, _ = distill_oracle(z, [1, 1, 0], [0.0, 0.0, np.log(2.0)], 1.0, 1.0)
    assert np.allclose(target, [0.5, 0.5, 0.0], atol=1e-15)
    for ids, t in (([-1, 3], [0.0, 0.0]), ([0, 1], [-np.inf, -np.inf])):
        assert distill_oracle(z, ids, t, 1.0, 1.0)[:2] == (0.0, 0.0)


def test_policy_by_hand():
    z = np.log(np.array([0.25, 0.75]))
    # ratio 1.5, above the border: clipped for A > 0, not for A < 0
    old = np.log(0.5)
    loss, lp, coef, q, target, _ = policy_oracle(z, 1, old, None, 2.0, 1.0, 0.2, 0.2, 0.0, 1.0)
    assert np.isclose(loss, -2.4) and coef == 0 and np.isclose(lp, np.log(0.75))
    loss, _, coef, q, target, _ = policy_oracle(z, 1, old, None, -2.0, 1.0, 0.2, 0.2, 0.0, 1.0)
    assert np.isclose(loss, 3.0) and np.isclose(coef, -3.0)
    # the KL term alone, ref / policy = 2
    loss, _, coef, _, _, _ = policy_oracle(z, 0, 0.0, np.log(0.5), 0.0, 1.0, 0.2, 0.2, 0.5, 1.0)
    assert np.isclose(loss, 0.5 * (2 - np.log(2) - 1)) and np.isclose(coef, 0.5)


@pytest.mark.parametrize("tau", [1.0, 0.6, 2.0])
def test_gradients(tau):
    rng = np.random.default_rng(3)
    for _ in range(20):
        z, ids, t = rng.standard_normal(9) * 2, rng.integers(-1, 10, 5), rng.standard_normal(5)
        w, old, ref, a = 0.7, -2.0 + rng.standard_normal(), -2.0 + rng.standard_normal(), rng.standard_normal()
        tok = int(rng.integers(0, 9))
        for f in (lambda x: distill_oracle(x, ids, t, w, tau),
                  lambda x: policy_oracle(x, tok, old, ref, a, w, 0.2, 0.3, 0.1, tau)):
            out = f(z)
            coef, q, target = (out[1:4] if len(out) == 5 else out[2:5])
            h = 1e-6
            diff = [(f(z + h * e)[0] - f(z - h * e)[0]) / (2 * h) for e in np.eye(9)]
            # a difference is off by some 1e-16 |f| / h
            assert np.allclose(coef * (q - target), diff, rtol=0, atol=1e-8 * (1 + abs(out[0])))
        # and torch's, from the definitions
        x = torch.tensor(z, requires_grad=True)
        lq = torch.log_softmax(x / tau, 0)
        there = [j for j in range(5) if 0 <= ids[j] < 9]
        if there:
            p = torch.softmax(torch.tensor(t[there]) / tau, 0)
            loss = w * tau ** 2 * (p * (p.log() - lq[ids[there]])).sum()
            g, = torch.autograd.grad(loss, x, retain_graph=True)
            out = distill_oracle(z, ids, t, w, tau)
            assert np.isclose(out[0], loss.item(), atol=1e-13)
            assert np.allclose(out[1] * (out[2] - out[3]), g.numpy(), atol=1e-13)
        r = torch.exp(lq[tok] - old)
        d = ref - lq[tok]
        loss = w * (-torch.minimum(r * a, r.clamp(0.8, 1.3) * a) + 0.1 * (torch.exp(d) - d - 1))
        g, = torch.autograd.grad(loss, x)
        out = policy_oracle(z, tok, old, ref, a, w, 0.2, 0.3, 0.1, tau)
        assert np.isclose(out[0], loss.item(), atol=1e-13)
        assert np.allclose(out[2] * (out[3] - out[4]), g.numpy(), atol=1e-13)

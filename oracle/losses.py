"""Oracle O8: the losses over a vocabulary's logits, row by row in 64 bits.
TEST INFRASTRUCTURE ONLY.

Each returns what a row gives besides the gradient: the probabilities q, the
target that is subtracted from them and the multiple of the difference
(gradient = coef * (q - target)), so that a test can bound each part's error.
"""

import numpy as np


def softmax_oracle(z, tau):
    """(q, log q) of a row that has a finite logit; logits of -inf have 0."""
    x = np.asarray(z, np.float64) / tau
    with np.errstate(invalid="ignore"):
        x = x - x.max()
        e = np.exp(x)
        s = e.sum()
        return e / s, x - np.log(s)


def distill_oracle(z, ids, t, weight, tau):
    """(loss, coef, q, target, size): size bounds the loss's terms."""
    vocab = len(z)
    zero = np.zeros(vocab)
    there = [j for j in range(len(ids)) if 0 <= ids[j] < vocab and t[j] != -np.inf]
    if not there or weight == 0 or np.all(z == -np.inf):
        return 0.0, 0.0, zero, zero, 0.0
    q, log_q = softmax_oracle(z, tau)
    p, log_p = softmax_oracle([t[j] for j in there], tau)
    target, loss, size = np.zeros(vocab), 0.0, 0.0
    for k, j in enumerate(there):
        target[ids[j]] += p[k]
        if p[k] > 0 or p[k] != p[k]:
            loss += p[k] * (log_p[k] - log_q[ids[j]])
            size += p[k] * (abs(log_p[k]) + abs(log_q[ids[j]]))
    w = float(weight)
    return w * tau * tau * loss, w * tau, q, target, w * tau * tau * size


def policy_oracle(z, token, old, ref, advantage, weight, clip_low, clip_high, kl, tau):
    """(loss, logp, coef, q, target, slope): slope bounds how much the loss and
    the multiple change with logp."""
    vocab = len(z)
    zero = np.zeros(vocab)
    if not 0 <= token < vocab or np.all(z == -np.inf):
        return 0.0, 0.0, 0.0, zero, zero, 0.0
    q, log_q = softmax_oracle(z, tau)
    lp = log_q[token]
    r, a, w = np.exp(lp - float(old)), float(advantage), float(weight)
    held = min(max(r, 1 - clip_low), 1 + clip_high)
    loss = -min(r * a, held * a)
    d_lp = -r * a if r * a <= held * a else 0.0
    slope = abs(r * a)
    if kl:
        d = float(ref) - lp
        loss += kl * (np.exp(d) - d - 1)
        d_lp += kl * (1 - np.exp(d))
        slope += abs(kl) * (1 + np.exp(d))
    target = zero.copy()
    target[token] = 1.0
    if w == 0:
        return 0.0, lp, 0.0, q, target, 0.0
    return w * loss, lp, -w * d_lp / tau, q, target, abs(w) * slope

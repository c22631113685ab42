"""Helpers of the layer operators' GPU tests."""

import numpy as np
import torch

from oracle.layers import bf16_widen_oracle
from tests._gpu import DEV, to_dev

U = 2.0 ** -24                  # half a step of fp32, relative


def bf16_patterns(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(
        torch.int16).numpy().view(np.uint16)


def rows(values, bf16, pad=0, offset=0):
    """A device matrix whose rows lie ``pad`` elements apart, ``offset``
    elements into its allocation, and the float64 values it holds.  The gaps
    hold NaN."""
    v = np.asarray(values, np.float32)
    n, c = v.shape
    wide = np.full((n, c + pad), np.nan, np.float32)
    wide[:, :c] = v
    flat = to_dev(bf16_patterns(wide).ravel() if bf16 else wide.ravel(), offset) if n else torch.empty(
        0, dtype=torch.bfloat16 if bf16 else torch.float32, device=DEV)
    held = bf16_widen_oracle(bf16_patterns(v)) if bf16 else v
    return flat.view(n, c + pad)[:, :c], held.astype(np.float64).reshape(n, c)


def checkpoint(codes, scales):
    """Device tensors of an oracle's checkpoint."""
    return (torch.from_numpy(codes).to(DEV).view(torch.float8_e4m3fn),
            torch.from_numpy(scales).to(DEV))


def workspace(nbytes):
    """Exactly nbytes, filled with a pattern: its contents must not matter."""
    return torch.full((nbytes,), 0xA5, dtype=torch.uint8, device=DEV)


class Window:
    """A main_grad window with guards on both sides that must stay as they
    are."""

    def __init__(self, length, seed, offset=0):
        self.before = np.random.default_rng(seed).standard_normal(length).astype(np.float32)
        self.buf = torch.full((length + 64 + offset,), 7.5, device=DEV)
        self.grad = self.buf[32 + offset:32 + offset + length]
        self.grad.copy_(torch.from_numpy(self.before))

    def after(self):
        torch.cuda.synchronize()
        whole = self.buf.cpu().numpy()
        n = self.grad.numel()
        at = whole.size - 32 - n
        assert (whole[:at] == 7.5).all() and (whole[at + n:] == 7.5).all(), "wrote outside the window"
        return whole[at:at + n]


def check_window(win, place, grad, size, terms, first, written=None, what=""):
    """The window against the float64 gradient ``grad`` of a parameter whose
    element 0 lies ``place`` elements into it; ``size``: the sums of the terms'
    magnitudes, ``terms``: how many at most (per element, or one number).

    A sum of m fp32 terms in any order, each add off by at most 2^-23 of its
    result (the matrix cores may truncate), is within m * 2^-23 * size of the
    exact sum; the scaling and the add into the window are within 2^-24 of
    their results."""
    got = win.after().astype(np.float64)
    before = np.zeros(got.size) if first else win.before.astype(np.float64)
    want, tol = win.before.astype(np.float64), np.zeros(got.size)
    g, size = grad.reshape(-1), size.reshape(-1)
    m = np.broadcast_to(terms, grad.shape).reshape(-1)
    touched = np.ones(g.size, bool) if written is None else np.broadcast_to(
        written, grad.shape).reshape(-1)
    a, b = max(0, -place), min(g.size, got.size - place)
    if a < b:
        sel = np.zeros(got.size, bool)
        sel[a + place:b + place] = touched[a:b]
        inside = np.zeros(g.size, bool)
        inside[a:b] = touched[a:b]
        want[sel] = before[sel] + g[inside]
        tol[sel] = 1.001 * (m[inside] * 2 * U * size[inside] + U * np.abs(g[inside]) +
                            U * np.abs(want[sel])) + 2.0 ** -149
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {got.size} off, first at "
                           f"{int(np.flatnonzero(bad)[0])}: {got[bad][0]!r} for {want[bad][0]!r}")
    return got

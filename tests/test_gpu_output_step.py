"""A training step of a small model of experts through the library alone: rows
looked up in the partitions, the experts' products, the logits of a tied output
layer, a loss, and all gradients back into the window, against torch's autograd
in 64 bits; then the reduction and Adam, after which the loss is taken again
from the partitions they wrote."""

import numpy as np
import pytest

from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._layers import U, workspace  # noqa: E402

R, VOCAB, DIM, TOKENS, TOP = 4, 1000, 72, 300, 5
COUNTS = [170, 0, 130]
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
B = 2.0 ** -8       # half a step of bf16, relative


def _bf16(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")


class Step:
    def __init__(self, seed, distill):
        rng = np.random.default_rng(seed)
        self.distill = distill
        numels = [VOCAB * DIM] + [DIM * DIM] * len(COUNTS)
        self.plan = zr.zr_plan_buckets(numels, [0] * len(numels), [(R, 1)], 20000, align=8)
        self.total, self.padded, self.P, _ = zr.zr_plan_group_info(self.plan, 0)
        self.master = torch.zeros(self.padded, device="cuda")
        self.master[:self.total] = torch.from_numpy((rng.standard_normal(self.total) * 0.3).astype(np.float32)).cuda()
        self.params = self.master.bfloat16()
        self.parts = list(self.params.split(self.P))
        self.ids = torch.from_numpy(rng.integers(0, VOCAB, TOKENS)).cuda()
        f32 = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()  # noqa: E731
        self.weight = f32(rng.random(TOKENS) / TOKENS)
        if distill:
            self.targets = torch.from_numpy(rng.integers(0, VOCAB, (TOKENS, TOP))).cuda()
            self.targets[:20] = -1
            self.teacher = f32(rng.standard_normal((TOKENS, TOP)))
        else:
            self.targets = torch.from_numpy(rng.integers(0, VOCAB, TOKENS)).cuda()
            self.targets[:20] = -100
            self.old, self.adv = f32(-7 + rng.standard_normal(TOKENS)), f32(rng.standard_normal(TOKENS))

    def product(self, name, params, counts, x, y):
        query, call = getattr(zr, name + "_workspace"), getattr(zr, name)
        out, width = (y.shape[1], x.shape[1]) if name == "zr_linear_forward" else (x.shape[1], y.shape[1])
        n = query(self.plan, params, counts, out, width)
        call(self.plan, params, counts, self.parts, x, y, workspace=workspace(n) if n else None)
        return y

    def forward(self):
        self.x = _bf16(TOKENS, DIM)
        zr.zr_embedding_lookup(self.plan, 0, DIM, self.parts, self.ids, self.x)
        self.h = self.product("zr_linear_forward", [1, 2, 3], COUNTS, self.x, _bf16(TOKENS, DIM))
        self.logits = self.product("zr_linear_forward", [0], [TOKENS], self.h, _bf16(TOKENS, VOCAB))
        self.dlogits, self.loss = _bf16(TOKENS, VOCAB), torch.empty(TOKENS, device="cuda")
        nbytes = zr.zr_loss_workspace(TOKENS, VOCAB, TOP if self.distill else 1, torch.bfloat16)
        ws = workspace(nbytes) if nbytes else None
        if self.distill:
            zr.zr_distill_loss(self.logits, self.targets, self.teacher, self.weight, self.loss, self.dlogits,
                               temperature=2.0, workspace=ws)
        else:
            zr.zr_policy_loss(self.logits, self.targets, self.old, None, self.adv, self.weight, self.loss,
                              torch.empty_like(self.loss), self.dlogits, workspace=ws)
        return self.loss.double().sum().item()

    def backward(self, grad):
        dh = self.product("zr_linear_input_grad", [0], [TOKENS], self.dlogits, _bf16(TOKENS, DIM))
        dx = self.product("zr_linear_input_grad", [1, 2, 3], COUNTS, dh, _bf16(TOKENS, DIM))
        kept = {}
        for name, t in (("x", self.x), ("h", self.h)):
            kept[name] = zr.act_empty(TOKENS, DIM)
            zr.zr_act_quantize(t, *kept[name])
        items, at = [(0, self.dlogits, *kept["h"])], 0
        for k, c in enumerate(COUNTS):
            items.append((1 + k, dh[at:at + c], *(t[at:at + c] for t in kept["x"])))
            at += c
        zr.zr_ipg_accumulate_linear_first(self.plan, items, grad,
                                          workspace(zr.zr_ipg_linear_workspace(self.plan, items, 0, self.padded)))
        zr.zr_ipg_accumulate_embedding(
            self.plan, 0, DIM, self.ids, dx, grad,
            workspace(zr.zr_ipg_embedding_workspace(self.plan, 0, DIM, TOKENS, 0, self.padded)))
        self.dh, self.dx = dh, dx
        self.kept = {}
        for name in kept:
            back = torch.empty(TOKENS, DIM, device="cuda")
            zr.zr_act_dequantize(*kept[name], back)
            self.kept[name] = back.double().cpu()


@pytest.mark.parametrize("distill", [True, False])
def test_step_against_autograd(distill):
    s = Step(1, distill)
    got_loss = s.forward()
    grad = torch.full((s.padded,), float("nan"), device="cuda")
    grad[s.total:] = 0
    s.backward(grad)
    # the same in 64 bits; what the library rounds on its way forward, and the
    # checkpoints that the weights' gradients take, have the library's values
    p = s.params.double().cpu()[:s.total]
    E = p[:VOCAB * DIM].view(VOCAB, DIM).clone().requires_grad_()
    W = [p[VOCAB * DIM + k * DIM * DIM:][:DIM * DIM].view(DIM, DIM).clone().requires_grad_() for k in range(len(COUNTS))]

    class Kept(torch.autograd.Function):
        """x W^T, with the checkpoint's values in the weight's gradient and the
        library's in the output."""
        @staticmethod
        def forward(ctx, x, w, kept, value):
            ctx.save_for_backward(w, kept)
            return value.clone()

        @staticmethod
        def backward(ctx, g):
            w, kept = ctx.saved_tensors
            return g @ w, g.t() @ kept, None, None
    x = E[s.ids.cpu()]
    assert torch.equal(x.detach(), s.x.double().cpu())
    pieces, at = [], 0
    for w, c in zip(W, COUNTS):
        pieces.append(Kept.apply(x[at:at + c], w, s.kept["x"][at:at + c], s.h.double().cpu()[at:at + c]))
        exact = s.x.double().cpu()[at:at + c] @ w.detach().t()
        size = s.x.double().cpu()[at:at + c].abs() @ w.detach().abs().t()
        assert ((pieces[-1].detach() - exact).abs() <= 1.01 * (B * exact.abs() + DIM * 2 * U * size)).all()
        at += c
    h = torch.cat(pieces)
    z = Kept.apply(h, E, s.kept["h"], s.logits.double().cpu())
    exact = (h @ E.t()).detach()
    size = h.detach().abs() @ E.detach().abs().t()
    assert ((z.detach() - exact).abs() <= 1.01 * (B * exact.abs() + DIM * 2 * U * size)).all()
    h.retain_grad()
    z.retain_grad()
    x.retain_grad()
    t, w = s.targets.cpu(), s.weight.double().cpu()
    used = (t >= 0) if not distill else (t >= 0).any(1)
    if distill:
        log_q = torch.log_softmax(z / 2.0, 1)
        log_pt = torch.log_softmax(s.teacher.double().cpu() / 2.0, 1)
        loss = (w * 4.0 * (log_pt.exp() * (log_pt - log_q.gather(1, t.clamp(min=0)))).sum(1))[used].sum()
    else:
        lp = torch.log_softmax(z, 1).gather(1, t.clamp(min=0)[:, None])[:, 0]
        r, a = torch.exp(lp - s.old.double().cpu()), s.adv.double().cpu()
        loss = (-w * torch.minimum(r * a, r.clamp(0.8, 1.2) * a))[used].sum()
    loss.backward()
    assert abs(got_loss - loss.item()) <= 1e-4 * w.sum()
    # dlogits off by 2^-8 of itself and the softmax's error, 600 U at this
    # vocabulary; dh and dx by that and their own roundings and sums
    dz, dh, dx = z.grad, h.grad, x.grad
    e = B + 600 * U
    assert ((s.dlogits.double().cpu() - dz).abs() <= 1.01 * e * dz.abs() + 1200 * U * w[:, None] * 20).all()
    size_h = (dz.abs() + 1200 * U * w[:, None] * 20) @ E.detach().abs()
    assert ((s.dh.double().cpu() - dh).abs() <= 1.01 * (2 * e + VOCAB * 2 * U) * size_h).all()
    size_x, at = [], 0
    for m, c in zip(W, COUNTS):
        size_x.append(size_h[at:at + c] @ m.detach().abs())
        at += c
    size_x = torch.cat(size_x)
    off_x = 3 * e + (VOCAB + DIM) * 2 * U
    assert ((s.dx.double().cpu() - dx).abs() <= 1.01 * off_x * size_x).all()
    got = grad.double().cpu()[:s.total]
    size = torch.zeros(VOCAB, DIM, dtype=torch.float64)
    size.index_add_(0, s.ids.cpu(), size_x)
    size += (dz.abs() + 1200 * U * w[:, None] * 20).t() @ s.kept["h"].abs()
    off = 1.01 * (off_x + (2 * TOKENS + 4) * 2 * U)
    assert ((got[:VOCAB * DIM].view(VOCAB, DIM) - E.grad).abs() <= off * size).all()
    at = 0
    for k, (m, c) in enumerate(zip(W, COUNTS)):
        g = got[VOCAB * DIM + k * DIM * DIM:][:DIM * DIM].view(DIM, DIM)
        if c == 0:
            assert (g == 0).all()
        else:
            size = size_h[at:at + c].t() @ s.kept["x"][at:at + c].abs()
            assert ((g - m.grad).abs() <= off * size).all()
        at += c


def test_step_and_reduction():
    """Every replica's window reduced into the partitions, which the next step
    reads."""
    s = Step(2, True)
    s.forward()
    grads = []
    for _ in range(R):
        g = torch.empty(s.padded, device="cuda")
        g[s.total:] = 0
        s.backward(g)
        grads.append(g)
    m, v = torch.zeros(s.padded, device="cuda"), torch.zeros(s.padded, device="cuda")
    before = s.params.clone()
    zr.zr_reduce_scatter_adam(s.plan, 0, -1, -1, grads, s.master, m, v, s.params, step=1, **HP)
    assert torch.equal(s.params, s.master.bfloat16()) and not torch.equal(s.params, before)
    s.forward()
    flat = s.params.double()
    want = s.x.double() @ torch.zeros(DIM, DIM, device="cuda", dtype=torch.float64)
    at = 0
    for k, c in enumerate(COUNTS):
        w = flat[VOCAB * DIM + k * DIM * DIM:][:DIM * DIM].view(DIM, DIM)
        want[at:at + c] = s.x[at:at + c].double() @ w.t().contiguous()
        at += c
    assert torch.equal(s.x, s.params[:VOCAB * DIM].view(VOCAB, DIM)[s.ids])
    assert ((s.h.double() - want).abs() <= B * want.abs() + 1e-4).all()

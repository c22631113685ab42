"""The losses against their oracle in 64 bits.

Errors that the tolerances count (U: half a step of fp32, relative).  An
exponent (z - m) c has three roundings, c's among them, so 2^x is off by
3 U |x| ln 2 and the 2 U of the exponential.  Over a row the terms of the sum
add up to 3 U H + 2 U of it, H <= ln V their entropy, plus a U for each add on
a term's way: fewer than V / 256 in a lane's own sum and 200 behind that.  So q
is off by q U (3 |ln q| + 3 ln V + V / 256 + 210), and log q by the row's part of it.
A teacher's probability is off by U (3 |ln p| + 6), over a row's entries U (3 ln
top + 6) of the terms, and each term by 4 U; the sums of them are 64-bit.  The
policy's ratio and exp(d) - d - 1 are off by their argument's error and 8 U.
Gradients round once more to their type, and so do the losses to fp32."""

import numpy as np
import pytest

from oracle.losses import distill_oracle, policy_oracle
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._gpu import to_dev  # noqa: E402
from tests._layers import U, rows as device_rows, workspace  # noqa: E402

CLIP = dict(clip_low=0.2, clip_high=0.28)


class Case:
    """A call's tensors and their values; the gradient lies between guards."""

    def __init__(self, rng, rows, vocab, bf16, top=0, tau=1.0, masked=0.0, wide=True, pad=0, offset=0,
                 kl=0.0, weighted=True, in_place=False, grad=True, teacher_bf16=False, values=None, grad_pad=None):
        z = rng.standard_normal((rows, vocab)) * 2
        if vocab > 8:
            z[np.arange(rows), rng.integers(0, vocab, rows)] += 9
        if values is not None:
            values(z)
        self.top, self.tau, self.kl, self.bf16, self.vocab = top, tau, kl, bf16, vocab
        self.logits, self.z = device_rows(z, bf16, pad, offset)
        none = rng.random(rows) < masked
        if top:
            self.ids = rng.integers(0, vocab, (rows, top))
            self.ids[:, top // 2:] = np.where(rng.random((rows, top - top // 2)) < 0.3, -1, self.ids[:, top // 2:])
            self.ids[none] = vocab
            self.teacher, self.t = device_rows(rng.standard_normal((rows, top)) * 2, teacher_bf16, pad, offset)
        else:
            self.ids = np.where(none, -100, rng.integers(0, vocab, rows))
        self.ids_dev = torch.from_numpy(self.ids if wide else self.ids.astype(np.int32)).cuda()
        self.w = (rng.random(rows) / max(rows, 1)).astype(np.float32) if weighted else np.ones(rows, np.float32)
        self.old, self.ref, self.adv = (rng.standard_normal(rows).astype(np.float32) for _ in range(3))
        for i in range(rows):       # ratios around 1
            if not top and 0 <= self.ids[i] < vocab:
                lp = policy_oracle(self.z[i], self.ids[i], 0.0, None, 0.0, 1.0, 0.2, 0.2, 0.0, tau)[1]
                if np.isfinite(lp):
                    self.old[i] = lp + 0.2 * self.old[i]
                    self.ref[i] = lp + 0.3 * self.ref[i]
        self.weight = to_dev(self.w, 1) if weighted and rows else None
        self.loss = torch.full((rows,), 7.5, device="cuda")
        self.logp = torch.full((rows,), 7.5, device="cuda")
        self.dlogits, self.wide_grad = None, None
        if in_place:
            self.dlogits = self.logits
        elif grad:
            gp = pad if grad_pad is None else grad_pad
            self.wide_grad = torch.full((rows + 2, vocab + gp), 7.5, device="cuda",
                                        dtype=torch.bfloat16 if bf16 else torch.float32)
            self.dlogits = self.wide_grad[1:rows + 1, :vocab]
        nbytes = zr.zr_loss_workspace(rows, vocab, max(top, 1), self.logits.dtype)
        self.ws = workspace(nbytes) if nbytes else None
        self.per = [to_dev(x, 1) if rows else torch.empty(0, device="cuda") for x in (self.old, self.ref, self.adv)]

    def call(self, stream=None):
        if self.top:
            zr.zr_distill_loss(self.logits, self.ids_dev, self.teacher, self.weight, self.loss, self.dlogits,
                               temperature=self.tau, workspace=self.ws, stream=stream)
        else:
            zr.zr_policy_loss(self.logits, self.ids_dev, self.per[0], self.per[1] if self.kl else None, self.per[2],
                              self.weight, self.loss, self.logp, self.dlogits, kl=self.kl, temperature=self.tau,
                              workspace=self.ws, stream=stream, **CLIP)

    def check(self, only=None):
        torch.cuda.synchronize()
        V = self.vocab
        if self.wide_grad is not None:
            g = self.wide_grad.float()
            assert (g[0] == 7.5).all() and (g[-1] == 7.5).all() and (g[:, V:] == 7.5).all(), "wrote outside"
        loss, logp = self.loss.double().cpu().numpy(), self.logp.double().cpu().numpy()
        part = U * (3 * np.log(V) + V / 256 + 210)
        half = 2.0 ** -8 if self.bf16 else U
        for i in range(len(loss)) if only is None else only:
            z, w = self.z[i], self.w[i]
            if self.top:
                want, coef, q, target, size = distill_oracle(z, self.ids[i], self.t[i], w, self.tau)
                tol = part * abs(w) * self.tau ** 2 + (10 + 3 * np.log(self.top)) * U * size + U * abs(want)
                drift = 0.0
            else:
                want, lp, coef, q, target, slope = policy_oracle(
                    z, self.ids[i], self.old[i], self.ref[i], self.adv[i], w, CLIP["clip_low"],
                    CLIP["clip_high"], self.kl, self.tau)
                off = part + 3 * U * abs(lp)
                assert abs(logp[i] - lp) <= off + U * abs(lp), (i, logp[i], lp)
                r = np.exp(lp - float(self.old[i])) if target.any() else 0.0
                assert min(abs(r - 0.8), abs(r - 1.28)) > 2 * off * r or w == 0, "a row on the border"
                tol = 1.01 * (off + 8 * U) * slope + U * abs(want)
                drift = 1.01 * (off + 8 * U) * slope / self.tau
            assert abs(loss[i] - want) <= tol, (i, loss[i], want, tol)
            if self.dlogits is None:
                continue
            got = self.dlogits[i].double().cpu().numpy()
            g = coef * (q - target)
            with np.errstate(divide="ignore"):
                lnq = np.where(q > 0, np.abs(np.log(q)), 0)
                lnp = np.where(target > 0, np.abs(np.log(target)), 0)
            rel = q * (part + 3 * U * np.minimum(lnq, 100)) + target * (8 + 3 * np.log(max(self.top, 1)) + max(self.top, 1)) * U + target * 3 * U * lnp
            tol = 1.01 * (abs(coef) * rel + (drift if not self.top else drift * abs(coef)) * np.abs(q - target)
                          + half * np.abs(g)) + 2.0 ** -126 * (1 + abs(coef))
            bad = np.abs(got - g) > tol
            assert not bad.any(), (i, int(bad.sum()), got[bad][0], g[bad][0])


SIZES = [(1, 1), (3, 7), (2, 40), (5, 1000), (64, 1023), (130, 8192), (130, 8200), (200, 4099), (7, 50257),
         (1, 128256), (129, 33001), (64, 20001), (65, 20001)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_distill(rows, vocab, bf16):
    rng = np.random.default_rng(rows * 7 + vocab)
    for top, kw in ((1, dict(tau=2.0, wide=False)), (17, dict(masked=0.3, pad=3, offset=1, teacher_bf16=True)),
                    (65, dict(tau=0.5, weighted=False, in_place=True)), (5, dict(grad=False, masked=0.2))):
        c = Case(rng, rows, vocab, bf16, top=top, **kw)
        c.call()
        c.check(range(0, rows, max(1, rows // 12)))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_policy(rows, vocab, bf16):
    rng = np.random.default_rng(rows * 11 + vocab)
    for kw in (dict(kl=0.1, tau=0.7, wide=False), dict(masked=0.3, pad=3, offset=1, kl=0.02),
               dict(weighted=False, in_place=True), dict(grad=False, masked=0.2, kl=-0.1), dict(grad_pad=5)):
        c = Case(rng, rows, vocab, bf16, **kw)
        c.call()
        c.check(range(0, rows, max(1, rows // 12)))


def test_rows_of_every_workgroup_size_and_longer():
    """More rows than are cut into pieces, of 256, 512 and 1024 lanes, and rows
    that the lanes' registers do not hold."""
    rng = np.random.default_rng(5)
    for vocab, bf16 in ((30000, True), (50257, True), (100001, True), (140001, True), (20001, False), (70007, False)):
        for top in (0, 33):
            c = Case(rng, 300, vocab, bf16, top=top, masked=0.1, kl=0.05)
            c.call()
            c.check(range(0, 300, 37))


@pytest.mark.parametrize("rows", [3, 150])
def test_many_entries_and_repeated_ones(rows):
    rng = np.random.default_rng(6)
    for vocab, top in ((40000, 1024), (13, 300)):
        c = Case(rng, rows, vocab, True, top=top)
        c.call()
        c.check(range(0, rows, max(1, rows // 5)))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,vocab", [(6, 300), (6, 40000), (160, 1500)])
def test_masked_logits(rows, vocab, bf16):
    """-inf and the type's lowest value in some places, in all but one, in all."""
    low = float(torch.finfo(torch.bfloat16).min)

    def values(z):
        z[0, ::2] = -np.inf
        z[1, ::2] = low
        z[2, 1:] = -np.inf
        z[3, 1:] = low
        z[4, :] = -np.inf
        z[5, :] = low
    rng = np.random.default_rng(7)
    for top in (0, 4):
        c = Case(rng, rows, vocab, bf16, top=top, values=values)
        if top:
            c.ids[:6] = [[1, 3, 1, -1], [1, 3, 1, -1], [0, -1, -1, -1], [0, -1, -1, -1], [1, 2, 3, 4], [1, 2, 3, 4]]
        else:
            c.ids[:6] = [1, 1, 0, 0, 1, 1]
            c.old[:6] = [policy_oracle(c.z[i], c.ids[i], 0.0, None, 0.0, 1.0, 0.2, 0.2, 0.0, 1.0)[1] for i in range(6)]
            c.per[0].copy_(torch.from_numpy(c.old))
        c.ids_dev.copy_(torch.from_numpy(c.ids))
        c.call()
        c.check(list(range(6)) + [rows - 1])
        assert (c.dlogits[4] == 0).all() and c.loss[4] == 0


def test_masked_target_and_non_finite_values():
    rng = np.random.default_rng(8)

    def values(z):
        z[0, 5], z[1, 5], z[2, 5] = -np.inf, np.nan, np.inf
        z[3, 6] = np.nan
    for rows, vocab in ((5, 200), (5, 40000), (140, 300)):
        c = Case(rng, rows, vocab, False, values=values, kl=0.5)
        c.ids[:4] = [5, 7, 7, -1]
        c.ids_dev.copy_(torch.from_numpy(c.ids))
        c.call()
        loss, g = c.loss.cpu().numpy(), c.dlogits.cpu().numpy()
        assert c.logp[0] == -np.inf and loss[0] == np.inf
        assert np.isnan(loss[1]) and np.isnan(g[1]).all() and np.isnan(loss[2]) and np.isnan(g[2]).all()
        assert loss[3] == 0 and (g[3] == 0).all() and np.isfinite(g[4:]).all()
        d = Case(rng, rows, vocab, False, top=3, values=values)
        d.ids[:5] = [[5, 7, 9], [7, 8, 9], [7, 8, 9], [-1, vocab, -7], [1, 2, 3]]
        d.ids_dev.copy_(torch.from_numpy(d.ids))
        d.teacher[4] = torch.tensor([1.0, float("nan"), 2.0])
        d.call()
        loss, g = d.loss.cpu().numpy(), d.dlogits.cpu().numpy()
        assert loss[0] == np.inf and np.isfinite(g[0]).all()
        assert np.isnan(g[1]).all() and np.isnan(g[2]).all() and loss[3] == 0 and (g[3] == 0).all()
        assert np.isnan(loss[4]) and np.isnan(g[4, 1:4]).all() and np.isfinite(g[4, 4:]).all()
        # a teacher without a finite entry, and a weight of 0 where all is NaN
        d.teacher[4] = -float("inf")
        d.weight[1] = 0.0
        d.call()
        assert d.loss[4] == 0 and (d.dlogits[4] == 0).all() and d.loss[1] == 0 and (d.dlogits[1] == 0).all()


def test_no_rows():
    for top in (0, 3):
        c = Case(np.random.default_rng(0), 0, 100, True, top=top)
        c.call()
        torch.cuda.synchronize()


def test_weighted_rows_of_differences():
    """The gradient of the summed losses against differences of the losses."""
    rng = np.random.default_rng(9)
    for top in (0, 6):
        c = Case(rng, 3, 50, False, top=top, kl=0.1, tau=0.8)
        c.call()
        g = c.dlogits.double().cpu().numpy()
        for i, v in ((0, 3), (1, 49), (2, 0)):
            h, value = 2.0 ** -4, {}
            x = c.logits[i, v].item()
            for s in (-2, -1, 1, 2):
                c.logits[i, v] = x + s * h
                c.call()
                value[s] = c.loss.double().sum().item()
            c.logits[i, v] = x
            # off by h^4 / 30 of the fifth derivative (under 40 times the loss's
            # size here) and by the losses' roundings over h
            diff = (8 * (value[1] - value[-1]) - (value[2] - value[-2])) / (12 * h)
            size = max(abs(t) for t in value.values()) + c.w[i]
            if not top:   # not where a step crosses the clip's border
                r = np.exp(c.logp[i].item() - c.old[i])
                if min(abs(r - 0.8), abs(r - 1.28)) < 0.4:
                    continue
            assert abs(diff - g[i, v]) <= size * (40 * h ** 4 / 30 + 300 * U / h)


def test_two_streams_and_graphs():
    rng = np.random.default_rng(10)
    cases = [Case(rng, 9, 40000, True, top=8), Case(rng, 9, 40000, True, kl=0.1),
             Case(rng, 200, 9000, True, top=8), Case(rng, 200, 9000, False, kl=0.1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for s, c in zip(streams, cases):
        c.call(stream=s)
    for c in cases:
        c.check(range(0, len(c.loss), 8))
        eager = [t.clone() for t in (c.loss, c.logp, c.dlogits)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        for _ in range(3):
            for t in (c.loss, c.logp, c.dlogits):
                t.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager[::2], (c.loss, c.dlogits)))
            assert c.top or torch.equal(eager[1], c.logp)
            torch.randn(1000, device="cuda").sum().item()


def test_two_graphs_share_a_workspace():
    """Pieces, and rows taken from a counter: nothing outlives a call."""
    rng = np.random.default_rng(11)
    cases = [Case(rng, 9, 40000, True, top=8), Case(rng, 530, 70000, True, top=8, masked=0.3),
             Case(rng, 520, 33000, False, kl=0.1, masked=0.3)]
    ws = workspace(max(c.ws.numel() for c in cases))
    graphs = []
    for c in cases:
        c.ws = ws
        c.call()
        c.check(range(0, len(c.loss), 40))
        graphs.append((torch.cuda.CUDAGraph(), c.dlogits.clone(), c.loss.clone()))
        with torch.cuda.graph(graphs[-1][0]):
            c.call()
    for _ in range(3):
        for (g, dlogits, loss), c in zip(graphs, cases):
            c.dlogits.fill_(3.0)
            g.replay()
            assert torch.equal(dlogits, c.dlogits) and torch.equal(loss, c.loss)
            c.call()
            assert torch.equal(dlogits, c.dlogits) and torch.equal(loss, c.loss)
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Logits of more than 2^32 bytes, and a gradient of as many."""
    rows, vocab = 17000, 128256
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    rng = np.random.default_rng(11)
    last = Case(rng, 4, vocab, True, kl=0.1)
    z[-4:] = last.logits
    g = torch.empty_like(z)
    put = lambda t, fill: torch.cat([torch.full((rows - 4,), fill, device="cuda", dtype=t.dtype), t])  # noqa: E731
    loss, logp = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zr.zr_policy_loss(z, put(last.ids_dev, 5), put(last.per[0], 0.0), put(last.per[1], 0.0), put(last.per[2], 1.0),
                      put(last.weight, 1.0), loss, logp, g, kl=0.1,
                      workspace=workspace(zr.zr_loss_workspace(rows, vocab, 1, z.dtype)), **CLIP)
    last.loss.copy_(loss[-4:])
    last.logp.copy_(logp[-4:])
    last.dlogits.copy_(g[-4:])
    last.check()
    # a row's exact gradient adds up to 0 (its size depends on how far old and
    # ref lie off): each element is off by 2^-8 of it and 2 part of a row's
    # terms, and the sum by U an add
    part = U * (3 * np.log(vocab) + vocab / 256 + 210)
    for rows_of in g[:-4].split(1000):
        f = rows_of.float()
        assert (f.sum(1).abs() <= (2.0 ** -8 + 2 * part + vocab * U) * f.abs().sum(1)).all()


def test_refusals():
    z = torch.zeros(4, 10, device="cuda")
    f, t = torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    te = torch.zeros(4, 2, device="cuda")

    def refused(match, call, *args, **kw):
        with pytest.raises(zr.ZrError, match=match):
            call(*args, **kw)
    for bad, match in ((f[:3], "has shape"), (f.double(), "must be"), (torch.zeros(8, device="cuda")[::2], "contiguous"),
                       (f.cpu(), "device")):
        refused(match, zr.zr_policy_loss, z, t, bad, None, f, None, f, f)
        refused(match, zr.zr_policy_loss, z, t, f, None, bad, None, f, f)
        refused(match, zr.zr_policy_loss, z, t, f, None, f, bad, f, f)
        refused(match, zr.zr_policy_loss, z, t, f, None, f, None, bad, f)
        refused(match, zr.zr_distill_loss, z, ids, te, bad, f)
        refused(match, zr.zr_distill_loss, z, ids, te, None, bad)
    refused("tokens has shape", zr.zr_policy_loss, z, t[:3], f, None, f, None, f, f)
    refused("tokens must", zr.zr_policy_loss, z, t.short(), f, None, f, None, f, f)
    refused("kl needs", zr.zr_policy_loss, z, t, f, None, f, None, f, f, kl=0.1)
    refused("dlogits must", zr.zr_policy_loss, z, t, f, None, f, None, f, f, z.bfloat16())
    refused("dlogits has shape", zr.zr_distill_loss, z, ids, te, None, f, z[:3])
    refused("contiguous rows", zr.zr_distill_loss, z.t(), ids, te, None, f)
    refused("ids must", zr.zr_distill_loss, z, ids.short(), te, None, f)
    refused("teacher has shape", zr.zr_distill_loss, z, ids, te[:, :1], None, f)
    refused("teacher must", zr.zr_distill_loss, z, ids, te.half(), None, f)
    refused("top must", zr.zr_distill_loss, z, ids[:, :0], te[:, :0], None, f)
    refused("contiguous rows", zr.zr_distill_loss, z, ids[:1].expand(4, 2).t().t(), te, None, f)
    assert f.abs().max() == 0

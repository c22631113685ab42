"""Measured cases of the operators that a training step needs between the
embedding and the gradient window: the products of layers whose weights lie in
the ranks' partitions, grouped by expert (forward, and the gradient of their
input), and two losses over a vocabulary's logits with their gradients,
distillation from a teacher's top logits and the clipped policy loss with a KL
term.

``own = False`` computes each in plain torch operations in 32 bits (the
policy's log-probabilities in 64, since ratios lie next to the clip's borders);
``own = True`` makes the library's calls.  ``exact`` is the definition in 64
bits.
"""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one new token through GPT-2 small's tied output layer
        dict(name="forward one token", op="forward", n_out=50257, n_in=768, experts=1, rows=1,
             skew=0.0, in_major=False, lead=0, world=1, dtype="bf16"),
        # a few tokens of a decoding batch, each routed to two of eight experts
        dict(name="forward few tokens", op="forward", n_out=8192, n_in=2048, experts=8, rows=32,
             skew=1.0, in_major=False, lead=0, world=2, dtype="bf16"),
        # a micro-batch of 8192 tokens, each routed to two of eight experts
        dict(name="forward experts", op="forward", n_out=8192, n_in=2048, experts=8, rows=16384,
             skew=0.5, in_major=False, lead=0, world=2, dtype="bf16"),
        # the logits of 2048 positions over Llama-3-8B's vocabulary
        dict(name="forward logits", op="forward", n_out=128256, n_in=4096, experts=1, rows=2048,
             skew=0.0, in_major=False, lead=0, world=8, dtype="bf16"),
        # GPT-2 small's attention weights, stored input-major, an odd batch; the
        # weight starts off 16 bytes and its gradient's consumer wants fp32
        dict(name="input grad odd", op="input_grad", n_out=2304, n_in=768, experts=1, rows=1531,
             skew=0.0, in_major=True, lead=5, world=3, dtype="fp32"),
        # the experts' second product backwards over the same micro-batch
        dict(name="input grad experts", op="input_grad", n_out=2048, n_in=8192, experts=8,
             rows=16384, skew=0.5, in_major=False, lead=0, world=2, dtype="bf16"),
        # eight positions of one sequence, fp32 logits
        dict(name="distill few rows", op="distill", rows=8, vocab=50257, top=16, dtype="fp32",
             temperature=1.0, masked=0.0, grad=True),
        # a sequence of 1024 over an odd vocabulary, softened, a tenth of it padding
        dict(name="distill sequence", op="distill", rows=1024, vocab=50257, top=64, dtype="bf16",
             temperature=2.0, masked=0.1, grad=True),
        # a micro-batch of 8192 over the large vocabulary
        dict(name="distill micro-batch", op="distill", rows=8192, vocab=128256, top=32,
             dtype="bf16", temperature=1.0, masked=0.0, grad=True),
        # the log-probabilities and losses alone, as an evaluation takes them
        dict(name="policy evaluated", op="policy", rows=777, vocab=50257, dtype="fp32",
             temperature=0.7, masked=0.1, kl=0.1, grad=False),
        # one short answer
        dict(name="policy one answer", op="policy", rows=64, vocab=128256, dtype="bf16",
             temperature=1.0, masked=0.0, kl=0.0, grad=True),
        # a batch of answers, prompts and padding masked
        dict(name="policy batch", op="policy", rows=4096, vocab=128256, dtype="bf16",
             temperature=1.0, masked=0.25, kl=0.02, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "input_grad", "input_grad", "distill", "policy"])
    if op in ("forward", "input_grad"):
        n_out, n_in = _log(rng, 64, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.6:
            n_out, n_in = -(-n_out // 64) * 64, -(-n_in // 64) * 64
        experts = min(rng.choice([1, 1, 2, 5, 8, 16]), max(1, 260_000_000 // (n_out * n_in)))
        rows = rng.choice([_log(rng, 1, 64), _log(rng, 1, 16384), _log(rng, 512, 16384)])
        rows = max(1, min(rows, 500_000_000_000 // (n_out * n_in)))
        return dict(op=op, n_out=n_out, n_in=n_in, experts=experts, rows=rows,
                    skew=rng.choice([0.0, 0.5, 1.0]), in_major=rng.random() < 0.4,
                    lead=rng.choice([0, 0, 3, 64]), world=rng.choice([1, 2, 3, 8]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    vocab = _log(rng, 1000, 160000)
    vocab += -vocab % 8 if rng.random() < 0.5 else 0
    case = dict(op=op, rows=min(_log(rng, 1, 8192), 400_000_000 // vocab), vocab=vocab,
                dtype=rng.choice(["bf16", "bf16", "fp32"]), temperature=rng.choice([0.7, 1.0, 2.0]),
                masked=rng.choice([0.0, 0.1, 0.5]), grad=rng.random() < 0.8)
    if op == "distill":
        case["top"] = _log(rng, 1, 256)
    else:
        case["kl"] = rng.choice([0.0, 0.02, 0.1])
    return case


# ------------------------------------------------------------------ inputs

CLIP = (0.2, 0.28)      # how far below and above 1 the policy's ratios count


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, sigma):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    return out.normal_(0.0, sigma, generator=gen)


def _counts(case):
    """Rows of each expert: shares that fall as (k + 1)^-skew, dealt out to the
    experts in a fixed mixed order, the last one's rounded down to none where
    there are few rows."""
    n, e = case["rows"], case["experts"]
    share = [(k + 1.0) ** -case["skew"] for k in range(e)]
    ends = [int(n * sum(share[:k + 1]) / sum(share) + 0.5) for k in range(e)]
    counts = [b - a for a, b in zip([0] + ends, ends)]
    step = next(s for s in (3, 5, 7) if e % s)
    return [counts[k * step % e] for k in range(e)]


def _products(case):
    lead = [case["lead"]] if case["lead"] else []
    numels = lead + [case["n_out"] * case["n_in"]] * case["experts"]
    return numels, len(lead), -(-sum(numels) // case["world"])


def _logits(gen, case):
    """Logits with a few high ones in each row, as a trained model's are."""
    rows, vocab = case["rows"], case["vocab"]
    z = _normal(gen, (rows, vocab), _dtype(case), 2.0)
    at = torch.randint(vocab, (rows, 8), generator=gen, device=DEV)
    z.scatter_(1, at, _normal(gen, (rows, 8), torch.float32, 3.0).add_(12.0).to(z.dtype))
    return z, at


def _rowwise(z, step, f):
    return torch.cat([f(z[i:i + step], slice(i, i + step)) for i in range(0, z.shape[0], step)])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=case)
    rows = case["rows"]
    if case["op"] in ("forward", "input_grad"):
        numels, first, part = _products(case)
        wide, narrow = ((case["n_in"], case["n_out"]) if case["op"] == "forward" else
                        (case["n_out"], case["n_in"]))
        s["flat"] = _normal(gen, part * case["world"], torch.bfloat16, 0.02)
        s["x"] = _normal(gen, (rows, wide), torch.bfloat16, 1.0)
        s["counts"] = _counts(case)
        if own:
            from zero_partition_aware_amd import zr
            s["zr"] = zr
            s["plan"] = zr.zr_plan_buckets(numels, [0] * len(numels), [(case["world"], 1)],
                                           500_000_000)
            s["parts"] = list(s["flat"].split(part))
            s["params"] = list(range(first, len(numels)))
            s["y"] = torch.empty(rows, narrow, dtype=_dtype(case), device=DEV)
            query = (zr.zr_linear_forward_workspace if case["op"] == "forward" else
                     zr.zr_linear_input_grad_workspace)
            s["workspace"] = torch.empty(
                query(s["plan"], s["params"], s["counts"], case["n_out"], case["n_in"],
                      in_major=case["in_major"]), dtype=torch.uint8, device=DEV)
        return s
    s["logits"], at = _logits(gen, case)
    keep = torch.rand(rows, generator=gen, device=DEV) >= case["masked"]
    s["weight"] = torch.full((rows,), 1.0 / rows, device=DEV)
    if case["op"] == "distill":
        # the teacher's entries: the student's own high ones and others
        top = case["top"]
        ids = torch.randint(case["vocab"], (rows, top), generator=gen, device=DEV)
        n = min(top, at.shape[1])
        ids[:, :n] = at[:, :n]
        teacher = _normal(gen, (rows, top), torch.float32, 2.0)
        teacher[:, :n] += 10.0
        ids[~keep] = -1
        s["ids"], s["teacher"] = ids.int(), teacher
    else:
        tokens = torch.where(torch.rand(rows, generator=gen, device=DEV) < 0.8, at[:, 0],
                             torch.randint(case["vocab"], (rows,), generator=gen, device=DEV))
        logp = _logp(s["logits"], tokens, case["temperature"])
        s["old"] = logp + _normal(gen, (rows,), torch.float32, 0.2)
        s["ref"] = logp + _normal(gen, (rows,), torch.float32, 0.3) if case["kl"] else None
        s["advantage"] = _normal(gen, (rows,), torch.float32, 1.0)
        s["tokens"] = torch.where(keep, tokens, -100)
    if own:
        from zero_partition_aware_amd import zr
        s["zr"] = zr
        s["loss"] = torch.empty(rows, device=DEV)
        s["logp"] = torch.empty(rows, device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"]) if case["grad"] else None
        s["workspace"] = torch.empty(
            zr.zr_loss_workspace(rows, case["vocab"], case.get("top", 1), s["logits"].dtype),
            dtype=torch.uint8, device=DEV)
    return s


def _logp(logits, tokens, temperature):
    def some(z, at):
        z = z.float() / temperature
        return z.gather(1, tokens[at, None])[:, 0] - z.logsumexp(1)
    return _rowwise(logits, 512, some)


# --------------------------------------------------------- the plain forms

def _weights(s, case):
    """Each expert's [n_out, n_in] weight, a view of the flat parameters."""
    _, first, _ = _products(case)
    o, i, n = case["n_out"], case["n_in"], case["n_out"] * case["n_in"]
    at = case["lead"] if first else 0
    for k in range(case["experts"]):
        w = s["flat"][at + k * n:at + (k + 1) * n]
        yield w.view(i, o).t() if case["in_major"] else w.view(o, i)


def _product(s, case):
    y, at = [], 0
    for w, n in zip(_weights(s, case), s["counts"]):
        if n:
            x = s["x"][at:at + n].float()
            y.append((x @ (w.float().t() if case["op"] == "forward" else w.float())).to(_dtype(case)))
            at += n
    return torch.cat(y)


def _distill(s, case):
    tau, vocab, losses, grads = case["temperature"], case["vocab"], [], []
    for i in range(0, case["rows"], 1024):
        z, ids = s["logits"][i:i + 1024].float() / tau, s["ids"][i:i + 1024].long()
        t, w = s["teacher"][i:i + 1024] / tau, s["weight"][i:i + 1024]
        there = (ids >= 0) & (ids < vocab)
        some = there.any(1)
        ids = ids.clamp(0, vocab - 1)
        t = torch.where(there, t, -math.inf)
        top = torch.where(some, t.amax(1), 0.0)
        e = torch.exp(t - top[:, None])
        p = e / torch.where(some, e.sum(1), 1.0)[:, None]
        high = z.amax(1)
        x = torch.exp(z - high[:, None])
        total = x.sum(1)
        log_q = z.gather(1, ids) - (high + total.log())[:, None]
        log_p = t - (top + torch.where(some, e.sum(1), 1.0).log())[:, None]
        terms = torch.where(p > 0, p * (log_p - log_q), 0.0)
        losses.append(torch.where(some, w * tau * tau * terms.sum(1), 0.0))
        if case["grad"]:
            scale = torch.where(some, w * tau, 0.0)[:, None]
            g = (x / total[:, None]).scatter_add(1, ids, -p)
            grads.append((g * scale).to(s["logits"].dtype))
    return (torch.cat(losses), torch.cat(grads)) if case["grad"] else torch.cat(losses)


def _policy(s, case):
    tau, vocab, losses, logps, grads = case["temperature"], case["vocab"], [], [], []
    for i in range(0, case["rows"], 1024):
        z, a = s["logits"][i:i + 1024].float(), s["tokens"][i:i + 1024]
        there = (a >= 0) & (a < vocab)
        a = a.clamp(0, vocab - 1)
        high = z.amax(1)
        # 64 bits for the sums: ratios lie next to the clip's borders
        x = torch.exp((z - high[:, None]).double() / tau)
        total = x.sum(1)
        logp = (z.gather(1, a[:, None])[:, 0] - high).double() / tau - total.log()
        ratio = torch.exp(logp - s["old"][i:i + 1024].double())
        adv, w = s["advantage"][i:i + 1024].double(), s["weight"][i:i + 1024].double()
        lo, hi = 1.0 - CLIP[0], 1.0 + CLIP[1]
        loss = -torch.minimum(ratio * adv, ratio.clamp(lo, hi) * adv)
        cut = ((adv > 0) & (ratio > hi)) | ((adv < 0) & (ratio < lo))
        slope = torch.where(cut, 0.0, -adv * ratio)
        if s["ref"] is not None:
            d = s["ref"][i:i + 1024].double() - logp
            loss = loss + case["kl"] * (torch.expm1(d) - d)
            slope = slope - case["kl"] * torch.expm1(d)
        losses.append(torch.where(there, w * loss, 0.0).float())
        logps.append(torch.where(there, logp, 0.0).float())
        if case["grad"]:
            scale = torch.where(there, w * slope / tau, 0.0).float()[:, None]
            g = (x / total[:, None]).float().neg_()
            g.scatter_add_(1, a[:, None], torch.ones_like(g[:, :1]))
            grads.append((g * scale).to(s["logits"].dtype))
    out = (torch.cat(losses), torch.cat(logps))
    return out + (torch.cat(grads),) if case["grad"] else out


def run(state):
    case = state["case"]
    if not own:
        return dict(distill=_distill, policy=_policy).get(case["op"], _product)(state, case)
    zr = state["zr"]
    if case["op"] in ("forward", "input_grad"):
        call = zr.zr_linear_forward if case["op"] == "forward" else zr.zr_linear_input_grad
        call(state["plan"], state["params"], state["counts"], state["parts"], state["x"],
             state["y"], workspace=state["workspace"], in_major=case["in_major"])
        return state["y"]
    if case["op"] == "distill":
        zr.zr_distill_loss(state["logits"], state["ids"], state["teacher"], state["weight"],
                           state["loss"], state["dlogits"], workspace=state["workspace"],
                           temperature=case["temperature"])
        return (state["loss"], state["dlogits"]) if case["grad"] else state["loss"]
    zr.zr_policy_loss(state["logits"], state["tokens"], state["old"], state["ref"],
                      state["advantage"], state["weight"], state["loss"], state["logp"],
                      state["dlogits"], workspace=state["workspace"], clip_low=CLIP[0],
                      clip_high=CLIP[1], kl=case["kl"], temperature=case["temperature"])
    out = (state["loss"], state["logp"])
    return out + (state["dlogits"],) if case["grad"] else out


# ------------------------------------------------------- what a pass needs

def work(case):
    size, rows = (2 if case["dtype"] == "bf16" else 4), case["rows"]
    if case["op"] in ("forward", "input_grad"):
        o, i = case["n_out"], case["n_in"]
        used = sum(1 for n in _counts(case) if n)
        x, y = (i, o) if case["op"] == "forward" else (o, i)
        return dict(bytes=used * o * i * 2 + rows * (x * 2 + y * size), flops=2.0 * rows * o * i)
    kept = rows * (1 - case["masked"])
    once = case["vocab"] * size
    extra = rows * (case["top"] * 8 + 8 if case["op"] == "distill" else 32)
    return dict(bytes=kept * once + (rows * once if case["grad"] else 0) + extra,
                flops=kept * case["vocab"] * (8 if case["grad"] else 4))


# ------------------------------------------------------ exact, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("forward", "input_grad"):
        out, at = [], 0
        per = case["n_out"] * case["n_in"]
        start = case["lead"]
        for k, n in enumerate(s["counts"]):
            w = s["flat"][start + k * per:start + (k + 1) * per].double()
            # [n_out, n_in] whichever way it is stored
            w = (w.view(case["n_in"], case["n_out"]).t() if case["in_major"] else
                 w.view(case["n_out"], case["n_in"])).contiguous()
            x = s["x"][at:at + n].double()
            out.append(torch.mm(x, w.t().contiguous()) if case["op"] == "forward" else torch.mm(x, w))
            at += n
        return torch.cat(out)
    tau, rows, vocab = case["temperature"], case["rows"], case["vocab"]
    loss = torch.zeros(rows, dtype=torch.float64, device=DEV)
    logp = torch.zeros_like(loss)
    # the gradient in the logits' own 64 bits, a few rows at a time
    grad = (torch.zeros(rows, vocab, dtype=torch.float64, device=DEV) if case["grad"] else None)
    for i in range(0, rows, 256):
        here = slice(i, min(i + 256, rows))
        log_q = torch.log_softmax(s["logits"][here].double() / tau, 1)
        w = s["weight"][here].double()
        if case["op"] == "distill":
            ids = s["ids"][here].long()
            valid = (ids >= 0) & (ids < vocab)
            used = valid.any(1)
            t = (s["teacher"][here].double() / tau).masked_fill(~valid, -1e300)
            log_p = torch.log_softmax(t, 1)
            p = log_p.exp() * valid
            at = ids.clamp(0, vocab - 1)
            loss[here] = w * tau ** 2 * (p * (log_p.clamp(min=-1e4) - log_q.gather(1, at))).sum(1) * used
            if case["grad"]:
                target = torch.zeros_like(log_q).scatter_add_(1, at, p)
                grad[here] = (log_q.exp() - target) * (w * tau * used)[:, None]
            continue
        a = s["tokens"][here]
        used = (a >= 0) & (a < vocab)
        at = a.clamp(0, vocab - 1)[:, None]
        lp = log_q.gather(1, at)[:, 0]
        r = (lp - s["old"][here].double()).exp()
        adv = s["advantage"][here].double()
        border = torch.where(adv > 0, 1.0 + CLIP[1], 1.0 - CLIP[0])
        inside = torch.where(adv > 0, r <= border, (r >= border) | (adv == 0))
        value = -adv * torch.where(inside, r, border)
        slope = -adv * r * inside
        if s["ref"] is not None:
            back = (s["ref"][here].double() - lp).exp()
            value += case["kl"] * (back - 1 - (s["ref"][here].double() - lp))
            slope += case["kl"] * (1 - back)
        loss[here], logp[here] = w * value * used, lp * used
        if case["grad"]:
            hot = torch.zeros_like(log_q).scatter_(1, at, 1.0)
            grad[here] = (hot - log_q.exp()) * (w * slope * used / tau)[:, None]
    out = (loss,) if case["op"] == "distill" else (loss, logp)
    out = out + (grad,) if case["grad"] else out
    return out if len(out) > 1 else out[0]

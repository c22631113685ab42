"""Measured cases of the operators between a model's layers and the flat
gradient window: the embedding lookup from the ranks' partitions, its gradient
by sorted tokens into ``main_grad``, activation checkpoints in 8 bits (stored
and restored), and the weight gradients taken from them into ``main_grad``.

``own = False`` computes each in plain torch operations in 32 bits; ``own =
True`` makes the library's calls.  ``exact`` is the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 32          # activations that share one power-of-two scale
E_MIN = -110        # smallest scale exponent of a block
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one new token of one sequence, its row taken from the rank that holds it
        dict(name="lookup one token", op="lookup", vocab=128256, dim=4096, n=1, lead=0, world=8,
             dtype="bf16", scale=1.0, masked=0.0),
        # a micro-batch of 8 sequences of 1024, rows scaled by sqrt(dim)
        dict(name="lookup micro-batch", op="lookup", vocab=128256, dim=4096, n=8192, lead=0,
             world=8, dtype="bf16", scale=64.0, masked=0.0),
        # a short odd batch: fp32 gradients, rows cut by the partition's ends
        dict(name="embed short fp32", op="embed", vocab=50257, dim=1001, n=333, lead=37, world=3,
             part=1, dtype="fp32", scale=1.0, masked=0.0, micro=1),
        # GPT-2 small's table, the whole of it, a tenth of the batch padding
        dict(name="embed small model", op="embed", vocab=50257, dim=768, n=8192, lead=0, world=1,
             part=0, dtype="bf16", scale=1.0, masked=0.1, micro=1),
        # one rank's eighth of a large table, two micro-batches of 32768 tokens
        dict(name="embed rank share", op="embed", vocab=128256, dim=4096, n=32768, lead=0,
             world=8, part=0, dtype="bf16", scale=64.0, masked=0.0, micro=2),
        # an odd batch of fp32 activations, the last block of a row incomplete
        dict(name="store odd fp32", op="store", rows=777, cols=1000, dtype="fp32"),
        # a layer's input saved for the backward pass
        dict(name="store layer input", op="store", rows=8192, cols=4096, dtype="bf16"),
        # one row handed back
        dict(name="restore one row", op="restore", rows=1, cols=4096, dtype="bf16"),
        # the inner activations of a feed-forward block handed back
        dict(name="restore inner", op="restore", rows=8192, cols=14336, dtype="bf16"),
        # GPT-2 small's attention weights, stored input-major: few weights, many tokens
        dict(name="linear few weights", op="linear", items="768>2304@8192,768>768@8192", lead=5,
             world=1, part=0, micro=1),
        # a feed-forward weight of Llama-3-8B over one micro-batch of 8192
        dict(name="linear large", op="linear", items="14336x4096@8192", lead=0, world=1, part=0,
             micro=1),
        # a rank's share of experts that got unequal numbers of tokens, one of
        # them none, over two micro-batches
        dict(name="linear experts", op="linear",
             items="8192x2048@1531,2048x8192@1531,8192x2048@517,2048x8192@517,"
                   "8192x2048@0,2048x8192@0", lead=0, world=2, part=0, micro=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "embed", "store", "restore", "linear", "linear"])
    if op in ("lookup", "embed"):
        dim = _log(rng, 64, 8192)
        dim += dim % 8 if rng.random() < 0.5 else 0
        case = dict(op=op, vocab=min(_log(rng, 1000, 150000), 520_000_000 // dim), dim=dim,
                    n=min(_log(rng, 1, 32768), 130_000_000 // dim), lead=rng.choice([0, 3, 64]),
                    world=rng.choice([1, 2, 3, 8]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    scale=rng.choice([1.0, math.sqrt(dim)]), masked=rng.choice([0.0, 0.2, 0.6]))
        if op == "embed":
            # a window of at most 130e6 gradients; the later rows are the rarer ones
            case["world"] = max(case["world"], -(-case["vocab"] * dim // 130_000_000))
            case["n"] = max(case["n"], 8)
            case.update(part=rng.randrange(case["world"]) if case["n"] > 2000 else 0,
                        micro=rng.choice([1, 2]))
        return case
    if op in ("store", "restore"):
        cols = _log(rng, 32, 16384)
        return dict(op=op, rows=min(_log(rng, 1, 16384), 110_000_000 // cols), cols=cols,
                    dtype=rng.choice(["bf16", "fp32"]))
    arrow, count, items = rng.choice("x>"), rng.choice([1, 1, 2, 4]), []
    for _ in range(count):
        a, b = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            a, b = -(-a // 64) * 64, -(-b // 64) * 64
        rows = rng.choice([_log(rng, 1, 8192), _log(rng, 256, 8192)])
        items.append("%d%s%d@%d" % (a, arrow, b, min(rows, 230_000_000_000 // (a * b * count))))
    world = rng.choice([1, 1, 2, 5])
    return dict(op=op, items=",".join(items), lead=rng.choice([0, 1, 16]), world=world,
                part=rng.randrange(world), micro=rng.choice([1, 2]))


# ------------------------------------------------------------------ layout

def _items(case):
    """(outputs, inputs, tokens, input-major) of each weight."""
    got = []
    for text in case["items"].split(","):
        shape, rows = text.split("@")
        a, b = shape.replace(">", "x").split("x")
        got.append((int(b), int(a), int(rows), True) if ">" in shape else
                   (int(a), int(b), int(rows), False))
    return got


def _numels(case):
    lead = [case["lead"]] if case["lead"] else []
    if case["op"] == "linear":
        return lead + [o * i for o, i, _, _ in _items(case)]
    return lead + [case["vocab"] * case["dim"]]


def _window(case):
    """[first, end) of the rank's partition in the flat space, with padding."""
    part = -(-sum(_numels(case)) // case["world"])
    return case["part"] * part, (case["part"] + 1) * part


def _code_cols(cols):
    return -(-cols // BLOCK) * BLOCK


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, sigma):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    return out.normal_(0.0, sigma, generator=gen)


def _tokens(gen, case):
    """Token ids whose frequency falls with their rank, some of them masked."""
    u = torch.rand(case["n"], generator=gen, device=DEV, dtype=torch.float64)
    t = (torch.exp(u * math.log(case["vocab"] + 1)).long() - 1).clamp_(0, case["vocab"] - 1)
    if case["masked"]:
        t[torch.rand(case["n"], generator=gen, device=DEV) < case["masked"]] = -100
    return t


def _activations(gen, rows, cols, dtype):
    """Normal values whose spread differs from channel to channel."""
    x = torch.empty(rows, cols, device=DEV).normal_(generator=gen)
    spread = torch.empty(cols, device=DEV).normal_(generator=gen).exp_()
    return x.mul_(spread).to(dtype)


def _plan(case):
    from zero_partition_aware_amd import zr
    numels = _numels(case)
    return zr, zr.zr_plan_buckets(numels, [0] * len(numels), [(case["world"], 1)], 500_000_000)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "lookup":
        part = -(-sum(_numels(case)) // case["world"])
        s["flat"] = _normal(gen, part * case["world"], _dtype(case), 0.02)
        s["tokens"] = _tokens(gen, case)
        if own:
            s["zr"], s["plan"] = _plan(case)
            s["parts"] = list(s["flat"].split(part))
            s["out"] = torch.empty(case["n"], case["dim"], dtype=_dtype(case), device=DEV)
    elif case["op"] == "embed":
        s["batches"] = [(_tokens(gen, case), _normal(gen, (case["n"], case["dim"]), _dtype(case), 1e-3))
                        for _ in range(case["micro"])]
        if own:
            lo, hi = _window(case)
            zr, s["plan"] = _plan(case)
            s["zr"] = zr
            s["main_grad"] = torch.zeros(hi - lo, device=DEV)
            s["workspace"] = torch.empty(
                zr.zr_ipg_embedding_workspace(s["plan"], len(_numels(case)) - 1, case["dim"],
                                              case["n"], lo, hi - lo),
                dtype=torch.uint8, device=DEV)
    elif case["op"] == "store":
        s["x"] = _activations(gen, case["rows"], case["cols"], _dtype(case))
        if own:
            from zero_partition_aware_amd import zr
            s["zr"] = zr
            s["codes"], s["scales"] = zr.act_empty(case["rows"], case["cols"], DEV)
    elif case["op"] == "restore":
        x = _activations(gen, case["rows"], case["cols"], torch.float32)
        s["codes"], s["scales"] = _store(x)
        if own:
            from zero_partition_aware_amd import zr
            s["zr"] = zr
            s["out"] = torch.empty(case["rows"], case["cols"], dtype=_dtype(case), device=DEV)
    else:
        s["batches"] = [[(_normal(gen, (rows, n_out), torch.bfloat16, 1e-3),
                          *_store(_activations(gen, rows, n_in, torch.float32)))
                         for n_out, n_in, rows, _ in _items(case)]
                        for _ in range(case["micro"])]
        if own:
            lo, hi = _window(case)
            zr, s["plan"] = _plan(case)
            s["zr"] = zr
            s["main_grad"] = torch.zeros(hi - lo, device=DEV)
            first = len(_numels(case)) - len(_items(case))
            s["items"] = [[(first + k, dy, codes, scales, item[3]) for k, (item, (dy, codes, scales))
                           in enumerate(zip(_items(case), batch))] for batch in s["batches"]]
            s["workspace"] = torch.empty(
                max(zr.zr_ipg_linear_workspace(s["plan"], items, lo, hi - lo)
                    for items in s["items"]), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------- the plain forms

def _store(x):
    """8-bit codes and the scale bytes (exponent + 127) of each block: the
    smallest power of two that keeps the block's finite values within 448."""
    rows, cols = x.shape
    pitch = _code_cols(cols)
    v = torch.nn.functional.pad(x.float(), (0, pitch - cols)).view(rows, pitch // BLOCK, BLOCK)
    top = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, E_MIN).clamp_(min=E_MIN).int()
    inverse = ((127 - e) << 23).view(torch.float32)
    return ((v * inverse.unsqueeze(-1)).to(E4M3).view(rows, pitch), (e + 127).to(torch.uint8))


def _restore(codes, scales, cols):
    scale = (scales.int() << 23).view(torch.float32)
    v = codes.float().view(*scales.shape, BLOCK) * scale.unsqueeze(-1)
    return v.view(codes.shape)[:, :cols]


def _lookup(s, case):
    start = case["lead"]
    table = s["flat"][start:start + case["vocab"] * case["dim"]].view(case["vocab"], case["dim"])
    t = s["tokens"]
    valid = (t >= 0) & (t < case["vocab"])
    rows = table[t.clamp(0, case["vocab"] - 1)].float() * case["scale"]
    return torch.where(valid.unsqueeze(1), rows, 0.0).to(table.dtype)


def _embed_one(case, tokens, dy, lo, hi):
    """The window's elements of the table's gradient, and the places before
    and after it that belong to no row."""
    start, dim = case["lead"], case["dim"]
    a, b = max(lo, start) - start, min(hi, start + case["vocab"] * dim) - start
    if a >= b:
        return torch.zeros(hi - lo, device=DEV)
    r0, r1 = a // dim, -(-b // dim)
    valid = (tokens >= r0) & (tokens < r1)
    g = torch.zeros(r1 - r0, dim, device=DEV)
    g.index_add_(0, (tokens - r0).clamp(0, r1 - r0 - 1),
                 torch.where(valid.unsqueeze(1), dy.float(), 0.0))
    g = (g * case["scale"]).view(-1)[a - r0 * dim:b - r0 * dim]
    return torch.nn.functional.pad(g, (a + start - lo, hi - b - start))


def _linear_one(case, batch, lo, hi):
    grads = [torch.zeros(case["lead"], device=DEV)]
    grads += [(_restore(codes, scales, n_in).t() @ dy.float() if in_major else
               dy.float().t() @ _restore(codes, scales, n_in)).reshape(-1)
              for (n_out, n_in, _, in_major), (dy, codes, scales) in zip(_items(case), batch)]
    flat = torch.cat(grads)
    return torch.nn.functional.pad(flat[lo:hi], (0, hi - max(lo, min(hi, flat.numel()))))


def run(state):
    case = state["case"]
    if own:
        zr = state["zr"]
        if case["op"] == "lookup":
            zr.zr_embedding_lookup(state["plan"], 1 if case["lead"] else 0, case["dim"],
                                   state["parts"], state["tokens"], state["out"],
                                   scale=case["scale"])
            return state["out"]
        if case["op"] == "store":
            zr.zr_act_quantize(state["x"], state["codes"], state["scales"])
            return state["codes"], state["scales"]
        if case["op"] == "restore":
            zr.zr_act_dequantize(state["codes"], state["scales"], state["out"])
            return state["out"]
        lo = _window(case)[0]
        if case["op"] == "embed":
            param, call = (1 if case["lead"] else 0), zr.zr_ipg_accumulate_embedding_first
            for tokens, dy in state["batches"]:
                call(state["plan"], param, case["dim"], tokens, dy, state["main_grad"],
                     state["workspace"], window_base=lo, scale=case["scale"])
                call = zr.zr_ipg_accumulate_embedding
            return state["main_grad"]
        call = zr.zr_ipg_accumulate_linear_first
        for items in state["items"]:
            call(state["plan"], items, state["main_grad"], state["workspace"], window_base=lo)
            call = zr.zr_ipg_accumulate_linear
        return state["main_grad"]
    if case["op"] == "lookup":
        return _lookup(state, case)
    if case["op"] == "store":
        return _store(state["x"])
    if case["op"] == "restore":
        return _restore(state["codes"], state["scales"], case["cols"]).to(_dtype(case))
    lo, hi = _window(case)
    if case["op"] == "embed":
        return sum(_embed_one(case, t, dy, lo, hi) for t, dy in state["batches"])
    return sum(_linear_one(case, batch, lo, hi) for batch in state["batches"])


# ------------------------------------------------------- what a pass needs

def _expected_rows(case, r0, r1):
    """How many tokens of a batch, and how many different ones, lie in the
    rows [r0, r1), for the distribution of _tokens."""
    v = np.arange(r0, r1, dtype=np.float64)
    p = np.log((v + 2) / (v + 1)) / math.log(case["vocab"] + 1) * (1 - case["masked"])
    return case["n"] * p.sum(), -np.expm1(case["n"] * np.log1p(-p)).sum()


def work(case):
    size = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "lookup":
        row = case["dim"] * size
        _, rows = _expected_rows(case, 0, case["vocab"])
        return dict(bytes=case["n"] * (8 + row) + rows * row, flops=case["n"] * case["dim"])
    if case["op"] in ("store", "restore"):
        code = case["rows"] * _code_cols(case["cols"]) * (1 + 1 / BLOCK)
        return dict(bytes=case["rows"] * case["cols"] * size + code,
                    flops=2 * case["rows"] * case["cols"])
    lo, hi = _window(case)
    if case["op"] == "embed":
        dim = case["dim"]
        a = min(max(lo - case["lead"], 0), case["vocab"] * dim)
        b = min(max(hi - case["lead"], 0), case["vocab"] * dim)
        tokens, rows = _expected_rows(case, a // dim, -(-b // dim))
        return dict(bytes=case["micro"] * (case["n"] * 8 + tokens * dim * size) + (b - a) * 4
                    + (case["micro"] - 1) * rows * dim * 8,
                    flops=case["micro"] * tokens * dim)
    # the share of each weight's rows that lies in the window
    need, flops, at = 0.0, 0.0, case["lead"]
    for n_out, n_in, rows, in_major in _items(case):
        share = max(0, min(hi, at + n_out * n_in) - max(lo, at)) / (n_out * n_in)
        dy, x = rows * n_out * 2, rows * _code_cols(n_in) * (1 + 1 / BLOCK)
        need += case["micro"] * ((dy + x * share if in_major else dy * share + x) * (share > 0))
        need += share * n_out * n_in * 4 * (2 * case["micro"] - 1)
        flops += case["micro"] * share * 2.0 * rows * n_out * n_in
        at += n_out * n_in
    return dict(bytes=need, flops=flops)


# ------------------------------------------------------ exact, in 64 bits

def _power(e):
    """2.0 ** e of whole numbers, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_store(x):
    rows, cols = x.shape
    v = torch.zeros(rows, _code_cols(cols), dtype=torch.float64, device=DEV)
    v[:, :cols] = x
    v = v.view(rows, -1, BLOCK)
    top = v.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -160) / 448)).clamp(min=E_MIN)
    e = torch.where((e > E_MIN) & (448 * _power(e - 1) >= top), e - 1, e)
    e = torch.where(448 * _power(e) < top, e + 1, e)
    v = v * _power(-e).unsqueeze(-1)
    # a code has 3 bits after its leading one, and steps of 2^-9 below 2^-6
    step = _power((torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3))
    return (torch.round(v / step) * step).view(rows, -1), (e + 127).to(torch.uint8)


def _exact_restore(codes, scales, cols):
    bits = codes.view(torch.uint8).long()
    e, m = (bits >> 3) & 15, bits & 7
    v = torch.where(e > 0, (8 + m) * _power(e - 10), m * _power(torch.full_like(e, -9)))
    v = torch.where(bits >= 128, -v, v).view(*scales.shape, BLOCK)
    return (v * _power(scales.long() - 127).unsqueeze(-1)).view(codes.shape)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(s["x"])
    if case["op"] == "restore":
        return _exact_restore(s["codes"], s["scales"], case["cols"])
    if case["op"] == "lookup":
        dim, t = case["dim"], s["tokens"]
        inside = (0 <= t) & (t < case["vocab"])
        at = case["lead"] + torch.where(inside, t, 0).unsqueeze(1) * dim + torch.arange(dim, device=DEV)
        return s["flat"][at.view(-1)].double().view(-1, dim) * case["scale"] * inside.unsqueeze(1)
    lo, hi = _window(case)
    # gradients by their place in the flat space, then the window of them
    g = torch.zeros(hi - lo + 1, dtype=torch.float64, device=DEV)
    if case["op"] == "embed":
        place = torch.arange(case["dim"], device=DEV)
        for tokens, dy in s["batches"]:
            for i in range(0, case["n"], 4096):
                t = tokens[i:i + 4096]
                at = case["lead"] - lo + t.unsqueeze(1) * case["dim"] + place
                outside = (at < 0) | (at >= hi - lo) | (t < 0).unsqueeze(1)
                at = torch.where(outside, hi - lo, at)
                g.index_put_((at.view(-1),), dy[i:i + 4096].double().view(-1) * case["scale"],
                             accumulate=True)
        return g[:-1]
    for batch in s["batches"]:
        at = case["lead"]
        for (n_out, n_in, _, in_major), (dy, codes, scales) in zip(_items(case), batch):
            x = _exact_restore(codes, scales, n_in)
            w = dy.double().t() @ x
            w = (w.t() if in_major else w).reshape(-1)
            a, b = max(lo, at), min(hi, at + w.numel())
            if a < b:
                g[a - lo:b - lo] += w[a - at:b - at]
            at += w.numel()
    return g[:-1]

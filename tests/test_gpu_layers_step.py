"""The layer operators as a training step uses them, with the library's own
reduction: rows looked up in the partitions, activations checkpointed in 8
bits, gradients of two micro-batches put into every replica's window, reduced
into the partitions with Adam, and the next lookup from what Adam wrote."""

import numpy as np
import pytest

from oracle.adam import adam_oracle
from oracle.bf16 import bf16_rne_oracle
from oracle.layers import (bf16_widen_oracle, dequantize_oracle, embedding_grad_oracle,
                           linear_grad_oracle, lookup_oracle, quantize_oracle)
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._gpu import assert_bits_equal, host_f32, host_u16, to_dev  # noqa: E402
from tests._layers import U, bf16_patterns, workspace  # noqa: E402

R, VOCAB, DIM, OUT, TOKENS, SCALE = 4, 91, 72, 130, 200, 8.0
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)


def test_step():
    rng = np.random.default_rng(0)
    numels = [VOCAB * DIM, OUT * DIM]
    plan = zr.zr_plan_buckets(numels, [0, 0], [(R, 1)], 5000, align=4)
    total, padded, P, _ = zr.zr_plan_group_info(plan, 0)
    theta = (rng.standard_normal(padded) * 0.05).astype(np.float32)
    theta[total:] = 0
    master, m, v = to_dev(theta), torch.zeros(padded, device="cuda"), torch.zeros(padded, device="cuda")
    params = to_dev(bf16_patterns(theta))
    parts = list(params.split(P))
    weights = bf16_widen_oracle(host_u16(params))
    table = host_u16(params)[:numels[0]].reshape(VOCAB, DIM)
    W = weights[numels[0]:total].reshape(OUT, DIM)

    grads, want, bound = [], [], []
    for r in range(R):
        full = torch.full((padded,), float("nan"), device="cuda")
        full[total:] = 0
        g, tol = np.zeros(total), np.zeros(total)
        for mb in range(2):
            tokens = rng.integers(0, VOCAB, TOKENS)
            tokens[rng.random(TOKENS) < 0.1] = -100
            ids = torch.from_numpy(tokens).cuda()
            x = torch.empty(TOKENS, DIM, dtype=torch.bfloat16, device="cuda")
            zr.zr_embedding_lookup(plan, 0, DIM, parts, ids, x, scale=SCALE)
            codes, scales = zr.act_empty(TOKENS, DIM)
            zr.zr_act_quantize(x, codes, scales)
            back = torch.empty(TOKENS, DIM, device="cuda")
            zr.zr_act_dequantize(codes, scales, back)
            # loss = sum(r * y), y = x^ W^T: dy = r, dx = dy W
            dy = torch.from_numpy(rng.standard_normal((TOKENS, OUT)).astype(np.float32)).cuda().bfloat16()
            dx = (dy.float() @ torch.from_numpy(W.copy()).cuda()).bfloat16()
            wsl = workspace(zr.zr_ipg_linear_workspace(plan, [(1, dy, codes, scales)], 0, padded))
            wse = workspace(zr.zr_ipg_embedding_workspace(plan, 0, DIM, TOKENS, 0, padded))
            linear, embed = ((zr.zr_ipg_accumulate_linear, zr.zr_ipg_accumulate_embedding) if mb else
                             (zr.zr_ipg_accumulate_linear_first, zr.zr_ipg_accumulate_embedding_first))
            linear(plan, [(1, dy, codes, scales)], full, wsl)
            embed(plan, 0, DIM, ids, dx, full, wse, scale=SCALE)
            # the same from the definitions
            wx = lookup_oracle(table, tokens, SCALE, True)
            assert np.array_equal(host_u16(x), wx)
            wc, wsc = quantize_oracle(bf16_widen_oracle(wx))
            assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), wc)
            xh = dequantize_oracle(wc, wsc, DIM)
            assert np.array_equal(back.double().cpu().numpy(), xh)
            gw, sw = linear_grad_oracle(dy.double().cpu().numpy(), xh, False)
            ge, se, _ = embedding_grad_oracle(VOCAB, tokens, dx.double().cpu().numpy(), SCALE)
            g += np.concatenate([ge.ravel(), gw.ravel()])
            tol += 2 * U * (TOKENS + 2) * np.concatenate([se.ravel(), sw.ravel()]) + U * np.abs(g)
        got = host_f32(full)[:total].astype(np.float64)
        assert (np.abs(got - g) <= 1.001 * tol).all()
        grads.append(full)
        want.append(g)
        bound.append(tol)

    zr.zr_reduce_scatter_adam(plan, 0, -1, -1, grads, master, m, v, params, step=1, **HP)
    # the reduction and Adam are checked bit for bit on what the windows hold
    held = [host_f32(x) for x in grads]
    mean = held[0] / np.float32(R)
    for x in held[1:]:
        mean = mean + x / np.float32(R)
    z = np.zeros(padded, np.float32)
    w_th, _, _ = adam_oracle(mean, theta, z, z, step=1, **HP)
    assert_bits_equal(host_f32(master), w_th, "master")
    # and the next forward pass reads the rows that Adam wrote
    ids = torch.arange(VOCAB, dtype=torch.int32, device="cuda")
    x = torch.empty(VOCAB, DIM, dtype=torch.bfloat16, device="cuda")
    zr.zr_embedding_lookup(plan, 0, DIM, parts, ids, x)
    assert np.array_equal(host_u16(x).ravel(), bf16_rne_oracle(w_th[:numels[0]]))


def test_gradients_against_autograd():
    """The gradients of a small network's loss, by torch in 64 bits from the
    activations that the checkpoint stands for."""
    rng = np.random.default_rng(1)
    plan = zr.zr_plan_buckets([VOCAB * DIM, OUT * DIM], [0, 0], [(1, 1)], 1 << 30)
    n = VOCAB * DIM + OUT * DIM
    params = torch.from_numpy((rng.standard_normal(n) * 0.05).astype(np.float32)).cuda().bfloat16()
    ids = torch.from_numpy(rng.integers(0, VOCAB, TOKENS)).cuda()
    x = torch.empty(TOKENS, DIM, dtype=torch.bfloat16, device="cuda")
    zr.zr_embedding_lookup(plan, 0, DIM, [params], ids, x, scale=SCALE)
    codes, scales = zr.act_empty(TOKENS, DIM)
    zr.zr_act_quantize(x, codes, scales)
    back = torch.empty(TOKENS, DIM, device="cuda")
    zr.zr_act_dequantize(codes, scales, back)
    p = params.double().cpu()
    E = p[:VOCAB * DIM].view(VOCAB, DIM).requires_grad_()
    W = p[VOCAB * DIM:].view(OUT, DIM).clone().requires_grad_()
    target = torch.from_numpy(rng.integers(0, OUT, TOKENS))
    xe = E[ids.cpu()] * SCALE
    # straight through the checkpoint: its values forward, the identity backward
    y = (xe + (back.double().cpu() - xe).detach()) @ W.t()
    y.retain_grad()
    xe.retain_grad()
    torch.nn.functional.cross_entropy(y, target, reduction="sum").backward()
    dy, dx = y.grad.float().bfloat16().cuda(), xe.grad.float().bfloat16().cuda()
    grad = torch.empty(n, device="cuda")
    items = [(1, dy, codes, scales)]
    zr.zr_ipg_accumulate_linear_first(plan, items, grad,
                                      workspace(zr.zr_ipg_linear_workspace(plan, items, 0, n)))
    zr.zr_ipg_accumulate_embedding_first(
        plan, 0, DIM, ids, dx, grad, workspace(zr.zr_ipg_embedding_workspace(plan, 0, DIM, TOKENS, 0, n)),
        scale=SCALE)
    got = grad.double().cpu().numpy()
    want = np.concatenate([E.grad.numpy().ravel(), W.grad.numpy().ravel()])
    # dy and dx are rounded to bf16 (through fp32): 2^-8 + 2^-24 of each term
    xa = back.double().cpu().abs().numpy()
    sw = np.abs(y.grad.numpy()).T @ xa
    se, _, _ = embedding_grad_oracle(VOCAB, ids.cpu().numpy(), np.abs(xe.grad.numpy()), SCALE)
    size = np.concatenate([se.ravel(), sw.ravel()])
    assert (np.abs(got - want) <= (2.0 ** -8 + 2 * U * (TOKENS + 3)) * 1.01 * size).all()

"""Pins of oracle/layers.py: the 8-bit code's values and rounding by hand and
against torch's cast, and the gradients against central differences of the
loss they belong to."""

import numpy as np
import pytest

from oracle.layers import (E4M3, bf16_widen_oracle, dequantize_oracle, embedding_grad_oracle,
                           linear_grad_oracle, lookup_oracle, quantize_oracle)


def test_code_values_by_hand():
    for code, value in ((0x00, 0.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9), (0x08, 2.0 ** -6),
                        (0x38, 1.0), (0x39, 1.125), (0x7E, 448.0), (0xB8, -1.0), (0xFE, -448.0)):
        assert E4M3[code] == value
    assert np.isnan(E4M3[0x7F]) and np.isnan(E4M3[0xFF])


def test_codes_agree_with_torch():
    torch = pytest.importorskip("torch")
    values = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(values.double().numpy(), E4M3, equal_nan=True)
    rng = np.random.default_rng(0)
    x = rng.uniform(-448, 448, (64, 32)).astype(np.float32)
    x[:, 0] = 448.0                                     # scale 1
    x[:32] *= np.exp2(rng.uniform(-16, 0, (32, 32))).astype(np.float32)
    x[:32, 0] = 448.0
    codes, scales = quantize_oracle(x)
    assert (scales == 127).all()
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)


def test_scale_is_the_least_that_holds_the_block():
    x = np.zeros((6, 33), np.float32)
    x[0, 3] = 448.0
    x[1, 3] = np.nextafter(np.float32(448.0), np.float32(1e9))
    x[2, 3] = -448.0 * 2.0 ** -30
    x[3, 32] = 1.0
    x[4, :3] = (1.0, np.inf, np.nan)
    x[5, 0] = 1e-40
    codes, scales = quantize_oracle(x)
    assert codes.shape == (6, 64) and scales.shape == (6, 2)
    assert scales[:, 0].tolist() == [127, 128, 97, 17, 119, 17]
    assert scales[3, 1] == 119                          # 1 = 256 * 2^-8
    assert codes[4, 1] == 0x7F and codes[4, 2] == 0x7F and codes[4, 0] == 0x78
    assert (codes[:, 33:] == 0).all()
    back = dequantize_oracle(codes, scales, 33)
    assert back[0, 3] == 448 and back[3, 32] == 1 and back[5, 0] == 0


def test_a_checkpoint_is_within_half_a_step():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 70)) * np.exp(rng.standard_normal(70))).astype(np.float32)
    codes, scales = quantize_oracle(x)
    d = np.abs(dequantize_oracle(codes, scales, 70) - x.astype(np.float64))
    step = np.repeat(np.ldexp(2.0 ** -9, scales.astype(np.int64) - 127), 32, axis=1)[:, :70]
    assert (d <= np.maximum(2.0 ** -4 * np.abs(x), step / 2)).all()


def test_gradients_are_the_loss_differences():
    """loss = sum(r * (x W^T)) with x = scale * E[tokens]: linear in W and in
    E, so central differences are the derivative up to their rounding."""
    rng = np.random.default_rng(2)
    vocab, dim, out, scale = 5, 4, 3, 1.5
    tokens = [1, 3, 1, -100, 4, 1, 7]
    E, W = rng.standard_normal((vocab, dim)), rng.standard_normal((out, dim))
    r = rng.standard_normal((len(tokens), out))

    def loss(E, W):
        x = np.stack([E[t] * scale if 0 <= t < vocab else np.zeros(dim) for t in tokens])
        return (r * (x @ W.T)).sum(), x

    _, x = loss(E, W)
    gw, _ = linear_grad_oracle(r, x, False)
    gt, _ = linear_grad_oracle(r, x, True)
    ge, _, count = embedding_grad_oracle(vocab, tokens, r @ W, scale)
    assert np.array_equal(gw, gt.T) and count.tolist() == [0, 3, 0, 1, 1]
    for a, g in ((E, ge), (W, gw)):
        for i in np.ndindex(a.shape):
            d = np.zeros_like(a)
            d[i] = 0.5
            args = ((E + d, W), (E - d, W)) if a is E else ((E, W + d), (E, W - d))
            assert abs((loss(*args[0])[0] - loss(*args[1])[0]) - g[i]) < 1e-12


def test_lookup_by_hand():
    t = np.array([[1.0, -2.0], [3.0, 0.3]], np.float32)
    assert lookup_oracle(t, [1, -1, 0, 2], 2.0, False).tolist() == [
        [6.0, float(np.float32(0.3) * np.float32(2))], [0, 0], [2.0, -4.0], [0, 0]]
    b = np.array([[0x3F80, 0x3F81]], np.uint16)         # 1, 1 + 2^-7
    assert bf16_widen_oracle(b).tolist() == [[1.0, 1.0078125]]
    # 1.5 * (1 + 2^-7) = 1.51171875 lies between 1.5078125 and 1.515625: a tie, to even
    assert lookup_oracle(b, [0], 1.5, True).tolist() == [[0x3FC0, 0x3FC2]]

"""Oracle O7: the layer operators, in plain numpy loops and 64-bit arithmetic.
TEST INFRASTRUCTURE ONLY.

What a model's layers read from the partitions and add to the gradient buffer:
embedding lookup and gradient, 8-bit activation checkpoints, and the weight
gradients taken from them.  Roundings to the stored types are done by table or
by the bf16 oracle, apart from the library's way of doing them.
"""

import numpy as np

from .bf16 import bf16_rne_oracle

BLOCK = 32
E_MIN = -110


def _e4m3_value(code):
    """The value of an e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 15 with mantissa 7 is NaN, there are no infinities."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


E4M3 = np.array([_e4m3_value(c) for c in range(256)])
_MAGNITUDE = E4M3[:127]         # codes 0..126, ascending


def _nearest_code(v):
    """Code of the nearest e4m3 value, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_MAGNITUDE, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dh, dl = np.abs(_MAGNITUDE[hi] - a), np.abs(a - _MAGNITUDE[lo])
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize_oracle(x):
    """(codes, scale bytes) of float32 rows x; codes padded to whole blocks."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = np.zeros((rows, blocks * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, BLOCK)
    finite = np.isfinite(v)
    top = np.where(finite, np.abs(v), 0.0).max(-1) if rows else np.zeros((0, blocks))
    e = np.full(top.shape, E_MIN)
    while True:         # the least exponent that holds the block
        small = np.ldexp(448.0, e) < top
        if not small.any():
            break
        e += small
    scaled = np.where(finite, v, 0.0) * np.ldexp(1.0, -e)[..., None]
    codes = np.where(finite, _nearest_code(scaled), 0x7F).astype(np.uint8)
    return codes.reshape(rows, blocks * BLOCK), (e + 127).astype(np.uint8)


def dequantize_oracle(codes, scales, cols):
    """float64 values a checkpoint stands for."""
    rows, blocks = scales.shape
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    return (E4M3[codes].reshape(rows, blocks, BLOCK) * s[..., None]).reshape(
        rows, blocks * BLOCK)[:, :cols]


def bf16_widen_oracle(bits):
    """float32 values of bf16 patterns."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)


def lookup_oracle(table, tokens, scale, bf16):
    """rnd(scale * table[token]) per row; rows of ids outside the table are 0.
    table: float32 [vocab, dim], or bf16 patterns (uint16)."""
    w = bf16_widen_oracle(table) if bf16 else np.asarray(table, np.float32)
    out = np.zeros((len(tokens), w.shape[1]), np.float32)
    for i, t in enumerate(tokens):
        if 0 <= t < w.shape[0]:
            out[i] = w[t] * np.float32(scale)
    return bf16_rne_oracle(out) if bf16 else out


def embedding_grad_oracle(vocab, tokens, dy, scale):
    """(gradient, sum of magnitudes, tokens per row) of the [vocab, dim]
    table, in float64."""
    g = np.zeros((vocab, dy.shape[1]))
    size, count = np.zeros_like(g), np.zeros(vocab, np.int64)
    for i, t in enumerate(tokens):
        if 0 <= t < vocab:
            g[t] += dy[i].astype(np.float64)
            size[t] += np.abs(dy[i].astype(np.float64))
            count[t] += 1
    s = float(np.float32(scale))
    return g * s, size * abs(s), count


def linear_grad_oracle(dy, x, in_major):
    """(gradient, sum of magnitudes) of the weight, float64, as stored."""
    dy, x = dy.astype(np.float64), x.astype(np.float64)
    if in_major:
        return x.T @ dy, np.abs(x).T @ np.abs(dy)
    return dy.T @ x, np.abs(dy).T @ np.abs(x)

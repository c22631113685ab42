"""zr_act_quantize and zr_act_dequantize against the float64 oracle, bit for
bit: a code is one rounding of an exact quotient, a restored value none."""

import numpy as np
import pytest

from oracle.layers import bf16_widen_oracle, dequantize_oracle, quantize_oracle
from tests._lib import load

pytestmark = pytest.mark.gpu

zr = load()
torch = pytest.importorskip("torch")
from tests._gpu import to_dev  # noqa: E402
from tests._layers import checkpoint, rows  # noqa: E402


def _store(x, bf16, pad=0, offset=0):
    t, held = rows(x, bf16, pad, offset)
    codes, scales = zr.act_empty(*x.shape)
    codes.view(torch.uint8).fill_(0x55)
    zr.zr_act_quantize(t, codes, scales)
    torch.cuda.synchronize()
    return codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), held.astype(np.float32)


def _same(codes, scales, held):
    want_codes, want_scales = quantize_oracle(held)
    assert np.array_equal(scales, want_scales)
    nan = (want_codes & 0x7F) == 0x7F
    assert np.array_equal((codes & 0x7F) == 0x7F, nan)
    assert np.array_equal(codes[~nan], want_codes[~nan])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("r,c,pad,offset", [
    (1, 1, 0, 0), (1, 32, 0, 0), (3, 31, 1, 1), (5, 33, 0, 3), (2, 64, 8, 0), (7, 100, 0, 1),
    (130, 257, 5, 0), (1, 5000, 0, 0), (1000, 7, 0, 2), (64, 1024, 0, 0), (33, 4104, 0, 0),
])
def test_store(r, c, pad, offset, bf16):
    rng = np.random.default_rng(r * 10000 + c)
    x = rng.standard_normal((r, c)) * np.exp(3 * rng.standard_normal(c))
    _same(*_store(x, bf16, pad, offset))


def test_store_every_finite_bf16_value_as_the_largest_of_its_block():
    bits = np.arange(65536, dtype=np.uint16)
    x = bf16_widen_oracle(bits)
    x = np.where(np.isfinite(x), x, 0).astype(np.float32)
    block = np.zeros((65536, 32), np.float32)
    block[:, 0] = x
    frac = np.random.default_rng(1).uniform(-1, 1, (65536, 31)).astype(np.float32)
    with np.errstate(under="ignore"):
        block[:, 1:] = x[:, None] * frac
    codes, scales, held = _store(block, False)
    _same(codes, scales, held)


def test_store_ties_borders_and_special_values():
    """Values half way between two codes, at the scale's border, infinities,
    NaNs, zeros and subnormals, also next to ordinary neighbours."""
    rng = np.random.default_rng(2)
    e4m3 = np.sort(dequantize_oracle(np.arange(127, dtype=np.uint8)[None].repeat(1, 0)[:, :96],
                                     np.full((1, 3), 127, np.uint8), 96)[0])
    mid = (e4m3[1:] + e4m3[:-1]) / 2
    pool = np.concatenate([mid, -mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                           np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                           [448, 449, 1e30, -1e38, 3.4e38, 1e-40, -1e-45, 0.0, -0.0]])
    x = rng.choice(pool, (600, 96)).astype(np.float32)
    x[100:200] = rng.choice(np.concatenate([mid, -mid]), (100, 96))
    x[100:200, ::32] = 448.0
    special = rng.random((600, 96)) < 0.05
    special[:300] = False
    x[special] = rng.choice([np.inf, -np.inf, np.nan], int(special.sum()))
    x[500:510] = np.nan
    x[510:520] = 0.0
    codes, scales, held = _store(x, False)
    _same(codes, scales, held)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("r,c,pad", [(1, 1, 0), (2, 33, 1), (256, 32, 0), (9, 1000, 0), (3, 4096, 7),
                                     (1000, 5, 0)])
def test_restore(r, c, pad, bf16):
    rng = np.random.default_rng(r + c)
    blocks = -(-c // 32)
    codes = rng.integers(0, 256, (r, 32 * blocks)).astype(np.uint8)
    scales = rng.integers(17, 240, (r, blocks)).astype(np.uint8)
    buf = torch.full((r * (c + pad) + 8,), 7.5, device="cuda",
                     dtype=torch.bfloat16 if bf16 else torch.float32)
    out = buf[1:1 + r * (c + pad)].view(r, c + pad)[:, :c]
    zr.zr_act_dequantize(*checkpoint(codes, scales), out)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), dequantize_oracle(codes, scales, c),
                          equal_nan=True)
    whole = buf.float().cpu()
    assert whole[0] == 7.5 and (whole[1 + r * (c + pad):] == 7.5).all()
    if pad:
        assert (whole[1:1 + r * (c + pad)].view(r, c + pad)[:, c:] == 7.5).all()


def test_store_then_restore_is_within_half_a_step():
    """Half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its
    normal range."""
    x = torch.randn(200, 515, device="cuda") * torch.exp(torch.randn(515, device="cuda"))
    codes, scales = zr.act_empty(200, 515)
    zr.zr_act_quantize(x, codes, scales)
    out = torch.empty_like(x)
    zr.zr_act_dequantize(codes, scales, out)
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :515]
    d = (out.double() - x.double()).abs()
    assert (d <= torch.maximum(x.double().abs() * 2.0 ** -4, s * 2.0 ** -10)).all()


def test_nothing_to_store():
    codes, scales = zr.act_empty(0, 40)
    zr.zr_act_quantize(to_dev(np.zeros(0, np.float32)).view(0, 40), codes, scales)
    zr.zr_act_dequantize(codes, scales, torch.empty(0, 40, device="cuda"))

"""The grouped products' kernels run on the CPU under AddressSanitizer +
UndefinedBehaviorSanitizer: zr_product.hip compiled as C++ against
tests/native/emu_waves and driven through the C ABI by
tests/native/products_emu.cpp on random plans, weights cut by partitions, groups
of rows, strides and offsets.  Loads into LDS arrive only when they are waited
for."""

import os

import pytest

from tests import _emu

pytestmark = pytest.mark.skipif(not os.path.exists(_emu.CLANG), reason="ROCm clang++ not available")

SHAPES = ("Shape<256, 256, 2, 4, 64, 2>", "Shape<32, 128, 1, 4, 64, 4>")
REQUIRED = ([f"product_kernel<(anonymous namespace)::{s}, {c}, {d}>" for s in SHAPES
             for c in ("false", "true") for d in ("false", "true")] +
            [f"product_join_kernel<(anonymous namespace)::{s}>" for s in SHAPES])


def test_product_kernels_on_cpu_under_asan_ubsan(tmp_path):
    exe = _emu.build(tmp_path, ["zr_product.hip"], "products_emu")
    launched = _emu.run(exe, [("60", str(1000 * k)) for k in range(6)], "product")
    assert launched >= set(REQUIRED), set(REQUIRED) - launched

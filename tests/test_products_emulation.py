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

SHAPES = ("Shape<32, 128, 1, 4, 64, 4>", "Shape<64, 128, 1, 4, 64, 3>", "Shape<128, 128, 2, 2, 64, 2>",
          "Shape<256, 256, 2, 4, 64, 2>")
REQUIRED = ([f"{k}<(anonymous namespace)::{s}, {c}>" for k in ("product_kernel", "product_any_kernel")
             for s in SHAPES for c in ("false", "true")] +
            [f"product_join_kernel<(anonymous namespace)::{s}>" for s in SHAPES])


def test_product_kernels_on_cpu_under_asan_ubsan(tmp_path):
    # a chip of two compute units: every shape of tiles at sizes that are quick here,
    # and several tiles to a workgroup
    exe = _emu.build(tmp_path, ["zr_product.hip"], "products_emu", "-DZR_CUS=2")
    launched = _emu.run(exe, [("60", str(1000 * k)) for k in range(6)], "product")
    assert launched >= set(REQUIRED), set(REQUIRED) - launched

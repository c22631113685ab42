"""The losses' kernels run on the CPU under AddressSanitizer +
UndefinedBehaviorSanitizer: zr_loss.hip compiled as C++ against
tests/native/emu_waves and driven through the C ABI by
tests/native/losses_emu.cpp on random rows, strides, entries and masks, with
the gradient in a buffer of its own and over the logits."""

import os

import pytest

from tests import _emu

pytestmark = pytest.mark.skipif(not os.path.exists(_emu.CLANG), reason="ROCm clang++ not available")

REQUIRED = ([f"loss_stats_kernel<{t}>" for t in ("float", "unsigned short")] +
            [f"loss_piece_kernel<{t}, {k}>" for t in ("float", "unsigned short") for k in ("false", "true")] +
            [f"loss_row_kernel<{t}, {k}, 256, 4>" for t in ("float", "unsigned short")
             for k in ("false", "true")])


def test_loss_kernels_on_cpu_under_asan_ubsan(tmp_path):
    exe = _emu.build(tmp_path, ["zr_loss.hip"], "losses_emu", "-DZR_CUS=40")
    runs = [("1", str(-k)) for k in range(1, 13)] + [("60", str(100 * k)) for k in range(6)]
    launched = _emu.run(exe, runs, "loss")
    assert launched >= set(REQUIRED), set(REQUIRED) - launched
    for lanes in (256, 512, 1024):
        assert any(f"{lanes}, 16>" in k for k in launched)

"""Every kernel that takes a row of logits to a workgroup, of each number of
lanes, dtype and loss, run on the CPU as test_losses_emulation.py does, on rows
that fill or pass a workgroup's registers."""

import os

import pytest

from tests import _emu

pytestmark = pytest.mark.skipif(not os.path.exists(_emu.CLANG), reason="ROCm clang++ not available")

REQUIRED = {f"loss_row_kernel<{t}, {k}, {lanes}, 16>" for t in ("float", "unsigned short")
            for k in ("false", "true") for lanes in (256, 512, 1024)} | {"loss_begin_kernel"}


def test_every_row_kernel_on_cpu_under_asan_ubsan(tmp_path):
    exe = _emu.build(tmp_path, ["zr_loss.hip"], "losses_emu", "-DZR_CUS=40")
    launched = _emu.run(exe, [("1", str(-k)) for k in range(1, 61)], "loss")
    assert launched >= REQUIRED, REQUIRED - launched

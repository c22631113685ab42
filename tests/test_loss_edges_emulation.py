"""The losses' kernels at the ends of what their arguments may hold, run on the
CPU under AddressSanitizer + UndefinedBehaviorSanitizer: tests/native/
loss_edges_emu.cpp, a section of it to each test."""

import os
import subprocess

import pytest

from tests import _emu

pytestmark = pytest.mark.skipif(not os.path.exists(_emu.CLANG), reason="ROCm clang++ not available")


@pytest.fixture(scope="module")
def edges(tmp_path_factory):
    exe = _emu.build(tmp_path_factory.mktemp("edges"), ["zr_loss.hip"], "loss_edges_emu", "-DZR_CUS=40")

    def run(section):
        out = subprocess.run([exe, section], capture_output=True, text=True, env=_emu.ENV, timeout=300)
        assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-4000:]
        assert "loss edges ok" in out.stdout
    return run


def test_rows_of_weight_0(edges):
    edges("weights")


def test_references_far_from_the_policy(edges):
    edges("references")


def test_ratios_that_fp32_does_not_hold(edges):
    edges("ratios")


def test_rows_far_from_0(edges):
    edges("far")


def test_multiples_that_fp32_does_not_hold(edges):
    edges("multiples")

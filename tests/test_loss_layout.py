"""What the losses' kernels read as 16-byte vectors lies on 16 bytes in LDS: a
compilation of zr_loss.hip for the host that states it."""

import os
import subprocess

import pytest

from tests import _emu

pytestmark = pytest.mark.skipif(not os.path.exists(_emu.CLANG), reason="ROCm clang++ not available")

STATED = """
#include "zr_loss.hip"
template <bool kTeacher>
constexpr bool entries_on_16_bytes =
    alignof(Entries<kTeacher>) % 16 == 0 && sizeof(Entries<kTeacher>) % 16 == 0 &&
    offsetof(Entries<kTeacher>, id) % 16 == 0 && alignof(Shared<kTeacher, 4>) % 16 == 0;
static_assert(entries_on_16_bytes<true> && entries_on_16_bytes<false>, "a row's entries lie on 16 bytes");
"""


def test_entries_lie_on_16_bytes(tmp_path):
    src = tmp_path / "layout.cpp"
    src.write_text(STATED)
    out = subprocess.run([*_emu.BASE, "-fsyntax-only", str(src)], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-3000:]

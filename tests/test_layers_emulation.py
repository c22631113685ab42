"""The layer operators' kernels run on the CPU under AddressSanitizer +
UndefinedBehaviorSanitizer: the library's own sources (zr_embed.hip,
zr_linear.hip compiled as C++ against tests/native/emu_waves, which runs the
lanes of a workgroup as coroutines) driven through the C ABI by
tests/native/layers_emu.cpp on random plans, windows, ids, strides and offsets.
An access outside a buffer, a workspace or LDS, a vector access at an address
its type does not allow, lanes of a wave that part before an operation of the
whole wave, or an output that differs from a plain loop fails the run."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"
CSRC = os.path.join(ROOT, "zero_partition_aware_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang++ not available")

ENV = dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1",
           # lanes have stacks of their own: no second one for each
           ASAN_OPTIONS="detect_leaks=1:abort_on_error=1:verify_asan_link_order=0:"
                        "detect_stack_use_after_return=0")

BASE = [CLANG, "-std=c++17", "-g", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(NATIVE, "emu_waves"),
        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include"]
# pointer-overflow: a weight's element 0 may lie before the window
SANITIZED = ["-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize=pointer-overflow", "-fno-sanitize-recover=all", "-ffp-contract=off"]


def _build(tmp_path):
    units = [(os.path.join(CSRC, "zr_embed.hip"), SANITIZED), (os.path.join(CSRC, "zr_linear.hip"), SANITIZED),
             (os.path.join(CSRC, "zr_plan.cpp"), SANITIZED),
             # the coroutines and the plain loops
             (os.path.join(NATIVE, "emu_waves", "waves.cpp"), ["-O2"]),
             (os.path.join(NATIVE, "layers_emu.cpp"), ["-O2"])]
    objects = [str(tmp_path / f"{k}.o") for k in range(len(units))]

    def compile_unit(k):
        src, flags = units[k]
        subprocess.run([*BASE, *flags, "-x", "c++", "-c", src, "-o", objects[k]], check=True,
                       capture_output=True, text=True)

    with ThreadPoolExecutor(len(units)) as pool:
        list(pool.map(compile_unit, range(len(units))))
    exe = str(tmp_path / "layers_emu")
    subprocess.run([CLANG, "-fsanitize=address,undefined", *objects, "-o", exe], check=True,
                   capture_output=True, text=True)
    return exe


REQUIRED = ([f"lookup_kernel<{t}>" for t in ("float", "unsigned short")] +
            [f"embed_sort_kernel<{t}>" for t in ("int", "long")] +
            [f"embed_sum_kernel<{t}, {first}, {tiny}>" for t in ("float", "unsigned short")
             for first in ("false", "true") for tiny in ("false", "true")] +
            [f"act_{k}_kernel<{t}>" for k in ("quantize", "dequantize") for t in ("float", "unsigned short")] +
            [f"{k}_kernel<{b}>" for k in ("embed_join", "linear_join") for b in ("false", "true")] +
            [f"linear_kernel<{b}, {d}>" for b in ("false", "true") for d in ("false", "true")])


def test_layer_kernels_on_cpu_under_asan_ubsan(tmp_path):
    exe = _build(tmp_path)
    runs = [("1", "-2"), ("1", "-1"), ("100", "0"), ("100", "100"), ("100", "200"), ("100", "300")]

    def run(args):
        return subprocess.run([exe, *args], capture_output=True, text=True, env=ENV, timeout=600)

    with ThreadPoolExecutor(len(runs)) as pool:
        outs = list(pool.map(run, runs))
    launched = set()
    for args, out in zip(runs, outs):
        assert out.returncode == 0, f"seeds {args}:" + out.stdout[-2000:] + out.stderr[-4000:]
        assert f"layer emulation ok: {args[0]} cases" in out.stdout
        launched |= {m.group(1) for m in re.finditer(r"^launches \d+ (.*)$", out.stdout, re.M)}
    assert launched >= set(REQUIRED), set(REQUIRED) - launched

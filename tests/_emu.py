"""Builds and runs the drivers that put the library's kernels through the CPU
under AddressSanitizer + UndefinedBehaviorSanitizer."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"
CSRC = os.path.join(ROOT, "zero_partition_aware_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")

ENV = dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1",
           # lanes have stacks of their own: no second one for each
           ASAN_OPTIONS="detect_leaks=1:abort_on_error=1:verify_asan_link_order=0:"
                        "detect_stack_use_after_return=0")

BASE = [CLANG, "-std=c++17", "-g", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(NATIVE, "emu_waves"),
        "-I", NATIVE, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include"]
SANITIZED = ["-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=all", "-ffp-contract=off"]


def build(tmp_path, sources, driver, *flags):
    """The driver with the library's ``sources`` (of csrc), sanitized."""
    units = [(os.path.join(CSRC, s), [*SANITIZED, *flags]) for s in (*sources, "zr_plan.cpp")]
    # the coroutines and the plain loops
    units += [(os.path.join(NATIVE, "emu_waves", "waves.cpp"), ["-O2"]),
              (os.path.join(NATIVE, driver + ".cpp"), ["-O2"])]
    objects = [str(tmp_path / f"{k}.o") for k in range(len(units))]

    def compile_unit(k):
        src, flags = units[k]
        out = subprocess.run([*BASE, *flags, "-x", "c++", "-c", src, "-o", objects[k]],
                             capture_output=True, text=True)
        assert out.returncode == 0, out.stderr[-4000:]

    with ThreadPoolExecutor(len(units)) as pool:
        list(pool.map(compile_unit, range(len(units))))
    exe = str(tmp_path / driver)
    subprocess.run([CLANG, "-fsanitize=address,undefined", *objects, "-o", exe], check=True,
                   capture_output=True, text=True)
    return exe


def run(exe, runs, what):
    """Runs (cases, first seed) each and returns the kernels launched."""
    def one(args):
        return subprocess.run([exe, *args], capture_output=True, text=True, env=ENV, timeout=600)

    with ThreadPoolExecutor(min(len(runs), 6)) as pool:
        outs = list(pool.map(one, runs))
    launched = set()
    for args, out in zip(runs, outs):
        assert out.returncode == 0, f"seeds {args}:" + out.stdout[-2000:] + out.stderr[-4000:]
        assert f"{what} emulation ok: {args[0]} cases" in out.stdout
        launched |= {m.group(1) for m in re.finditer(r"^launches \d+ (.*)$", out.stdout, re.M)}
    return launched

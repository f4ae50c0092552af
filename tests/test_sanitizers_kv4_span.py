"""The attention's count of keys without the gap between first tokens and window, and the plan that
cuts it, under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ missing")
    exe = str(tmp_path_factory.mktemp("kv4") / "kv4_span_driver")
    cmd = [CLANG, "-x", "c++", "-std=c++17"] + SAN + \
        ["-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "block_wise_int4_amd", "csrc"), "-I/opt/rocm/include",
         "-D__HIP_PLATFORM_AMD__", os.path.join(ROOT, "tests", "sanitize", "kv4_span_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("part", ["blocks", "alone", "wide", "plans"])
def test_the_count_of_visible_keys(driver, part):
    r = subprocess.run([driver, part], capture_output=True, text=True, env=ENV, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok: 0 failures"), r.stdout[-2000:] + r.stderr[-3000:]

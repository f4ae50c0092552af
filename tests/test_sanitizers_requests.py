"""The argument checks and the plan of the adapters and the verification under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang++ missing")
def test_requests_calls_host_side_under_sanitizers(tmp_path):
    exe = str(tmp_path / "requests_api_driver")
    csrc = os.path.join(ROOT, "block_wise_int4_amd", "csrc")
    inc = ["-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__"]
    build = [CLANG, "-x", "c++", "-std=c++17"] + SAN + inc + \
        [os.path.join(csrc, "mnb_requests_api.cpp"), os.path.join(ROOT, "tests", "sanitize", "requests_api_driver.cpp"), "-o", exe,
         "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    for cmd in (build, [exe]):
        r = subprocess.run(cmd, cwd=ROOT, capture_output=True, text=True, env=ENV, timeout=300)
        assert r.returncode == 0, "%s\n%s\n%s" % (" ".join(cmd), r.stdout[-3000:], r.stderr[-3000:])
    assert r.stdout.strip().endswith("ok: 0 failures")

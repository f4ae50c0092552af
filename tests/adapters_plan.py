"""How a call of the adapters is cut, asked of the library's own plan on the host."""
import ctypes
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_wise_int4_amd", "csrc")
FIELDS = ("one", "splits", "k_per", "down_tile", "up_tile", "down_ranks", "one_slots", "down_slots", "up_slots", "up_blocks", "pitch")
Plan = namedtuple("Plan", FIELDS)
SOURCE = """
#include "adapters_plan.hpp"
extern "C" void plan(int64_t m, int64_t n, int64_t k, int rank, int count, int f16, int64_t* out)
{
    const mnb::adapters::Plan c = mnb::adapters::plan_of(m, n, k, rank, count, f16);
    int i = 0;
%s}
""" % "".join("    out[i++] = c.%s;\n" % f for f in FIELDS)


def build(folder):
    """plan_of(m, n, k, rank, count, f16) from the header, compiled into `folder`."""
    compiler = shutil.which("g++") or shutil.which("clang++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([compiler, "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, src, "-o", lib], check=True, timeout=120)
    call = ctypes.CDLL(lib).plan
    call.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int64)]
    call.restype = None

    def plan_of(m, n, k, rank, count, f16):
        out = (ctypes.c_int64 * len(FIELDS))()
        call(m, n, k, rank, count, int(f16), out)
        return Plan(*out)

    return plan_of

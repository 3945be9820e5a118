"""The host-side rules of the block-scaled fp8 products (csrc/fp8_rules.h), compiled
with g++ and called through ctypes: no GPU is needed."""
import ctypes as C
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tile_planned_generator_amd", "csrc")
SHIM = """
#include "fp8_rules.h"
extern "C" {
int experts_disjoint(int64_t M, int64_t N, int64_t ld, int64_t stride, int64_t experts)
{ return dg::experts_disjoint(M, N, ld, stride, experts); }
int rows_fit_32(int rows, int64_t ld, int64_t K) { return dg::rows_fit_32(rows, ld, K); }
}
"""


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, src, "-o", so], check=True)
        loaded = C.CDLL(so)
    loaded.experts_disjoint.argtypes = [C.c_int64] * 5
    loaded.rows_fit_32.argtypes = [C.c_int, C.c_int64, C.c_int64]
    return loaded

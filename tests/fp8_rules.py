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
int grid_fits(int64_t workgroups, int threads, int64_t times) { return dg::grid_fits((__int128)workgroups * times, threads); }
int rows_fit_32(int rows, int64_t ld, int64_t K) { return dg::rows_fit_32(rows, ld, K); }
int choose_dense(int64_t M, int64_t N, int64_t K, int exact, int64_t lda, int64_t ldb)
{ return dg::choose_dense(M, N, K, dg::huge_tile(exact, lda, ldb, K)).kernel; }
int choose_rows(int64_t rows, int64_t experts, int64_t N, int exact, int64_t lda, int64_t ldb)
{ return dg::choose_rows(rows, experts, N, exact, dg::huge_tile(exact, lda, ldb, 0)); }
int choose_wgrad(int64_t M, int64_t N, int64_t experts, int exact, int64_t lda, int64_t ldb)
{ return dg::choose_wgrad(M, N, experts, dg::huge_tile(exact, lda, ldb, 0)); }
}
"""
STREAM16, TILE64, TILE128, TILE256 = range(4)


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, src, "-o", so], check=True)
        loaded = C.CDLL(so)
    loaded.experts_disjoint.argtypes = [C.c_int64] * 5
    loaded.grid_fits.argtypes = [C.c_int64, C.c_int, C.c_int64]
    loaded.rows_fit_32.argtypes = [C.c_int, C.c_int64, C.c_int64]
    for choose in (loaded.choose_dense, loaded.choose_rows, loaded.choose_wgrad):
        choose.argtypes = [C.c_int64] * 3 + [C.c_int, C.c_int64, C.c_int64]
    return loaded


def dense(M, N, K, exact, lda=16, ldb=16):
    return lib().choose_dense(M, N, K, exact, lda, ldb)


def rows(n, experts, N, exact, lda=16, ldb=16):
    return lib().choose_rows(n, experts, N, exact, lda, ldb)


def wgrad(M, N, experts, exact, lda=16, ldb=16):
    return lib().choose_wgrad(M, N, experts, exact, lda, ldb)

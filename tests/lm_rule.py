"""The language-model products' choice of tiles (csrc/lm_rule.hpp, plain C++) on the host:
which kernels a call launches on a device of 256 compute units."""
import ctypes
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """#include <initializer_list>
#include "%s/fp32_gemm_04_amd/csrc/lm_rule.hpp"
using namespace sgemm::lm;
extern "C" int rows(int size, int fast, int64_t used, int64_t rows, int64_t N, int64_t K)
{
    return rows_tile(size, fast, used, rows, N, K, 256);
}
extern "C" int sum(int size, int fast, int groups, int rows, int64_t M, int64_t N)
{
    return sum_tile(size, fast, groups, rows, M, N, 256);
}
extern "C" int stats(int size, int fast, int64_t T, int64_t V, int64_t K)
{
    return plain_tile(size, F_STATS, fast, T, V, K, 256);
}
extern "C" void backward(int size, int fast_x, int fast_w, int T, int V, int K, int64_t *out)
{
    const XentPlan p = xent_plan(size, fast_w, T, V, K, 256);
    const int64_t last = V - (p.pieces - 1) * p.piece, most = p.pieces > 1 ? p.piece : last;
    int64_t *o = out;
    *o++ = p.pieces > 1, *o++ = p.slices > 1, *o++ = p.low_rows, *o++ = p.dx_form == F_DX, *o++ = p.dx_tile;
    for (int64_t n : {most, last}) {
        *o++ = grad_tile(size, fast_x && fast_w, p, T, n, K, 256);
        *o++ = plain_tile(size, F_DW, fast_x, n, K, p.d_rows, 256);
    }
}
"""
TILES = ("16", "32", "48", "64", "128", "192", "256")


def _load():
    with tempfile.TemporaryDirectory(prefix="lm_rule_") as d:
        source, lib = os.path.join(d, "rule.cpp"), os.path.join(d, "rule.so")
        with open(source, "w") as f:
            f.write(SOURCE % ROOT)
        subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", lib, source], check=True)
        lib = ctypes.CDLL(lib)
    i, l = ctypes.c_int, ctypes.c_int64
    lib.rows.argtypes = [i, i, l, l, l, l]
    lib.sum.argtypes = [i, i, i, i, l, l]
    lib.stats.argtypes = [i, i, l, l, l]
    lib.backward.argtypes = [i] * 6 + [ctypes.POINTER(l)]
    return lib


_lib = None


def lib():
    global _lib
    _lib = _lib or _load()
    return _lib


def grouped(size, fast, groups, rows, N, K):
    """The kernel of a grouped product with `rows` rows in all."""
    return {(size, fast, "rows", TILES[lib().rows(size, fast, min(groups, rows), rows, N, K)])}


def wgrad(size, fast, groups, rows, M, N):
    return {(size, fast, "sum", TILES[lib().sum(size, fast, groups, rows, M, N)])}


def xent(size, fast, T, V, K):
    """The kernels of a loss and its gradients."""
    o = (ctypes.c_int64 * 9)()
    lib().backward(size, fast, fast, T, V, K, o)
    pieces, slices, low, direct = o[:4]
    wrap = "wrap" if 0 < low < 64 else "wrap64" if low else ""
    out = {(size, fast, "stats", TILES[lib().stats(size, fast, T, V, K)]),
           (size, fast, "dx" if direct else "part", TILES[o[4]]),
           (size, fast, "sums", "of pieces" if pieces else "of one", "in slices" if slices else "whole")}
    for grad, dw in (o[5:7], o[7:9]):
        out |= {(size, fast, "grad", TILES[grad], "remainders" if low else ""),
                (size, fast, "dw", TILES[dw], wrap)}
    return out

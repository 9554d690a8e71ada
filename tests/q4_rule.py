"""The 4-bit products' choice of kernel (csrc/q4_rule.hpp, plain C++) on the host, for a
device of 256 compute units."""
import ctypes
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """#include "%s/fp32_gemm_04_amd/csrc/q4_rule.hpp"
extern "C" void plan(int size, int offsets, int groups, int rows, int64_t N, int64_t K, int block, int *out)
{
    const sgemm::q4::Q4Plan p = sgemm::q4::q4_plan(size, offsets, groups, rows, N, K, block, 256);
    const int values[] = {p.rt, p.nt, p.wn, p.cols, p.pass, p.slab_log2, p.lds};
    for (int i = 0; i < 7; ++i) out[i] = values[i];
}
"""
_lib = None


def plan(size, offsets, groups, rows, N, K, block):
    """rt, nt, wn, cols, pass, slab_log2, lds."""
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory(prefix="q4_rule_") as d:
            source, lib = os.path.join(d, "rule.cpp"), os.path.join(d, "rule.so")
            with open(source, "w") as f:
                f.write(SOURCE % ROOT)
            subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", lib, source], check=True)
            _lib = ctypes.CDLL(lib)
        _lib.plan.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] * 2 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    out = (ctypes.c_int * 7)()
    _lib.plan(size, offsets, groups, rows, N, K, block, out)
    return tuple(out)


def kernels(size, groups, rows, N, K, block):
    """What a product with one set of weights (groups 0) or several runs; rows of weights
    whose bytes divide by four take direct loads."""
    rt, nt, wn, _, pass_, slab_log2, _ = plan(size, groups > 0, max(groups, 1), rows, N, K, block)
    return {(size, "block", block, "form", rt, nt, "direct" if K % 8 == 0 else "registers"),
            (size, "form", rt, nt, "waves", wn),
            (size, "form", rt, nt, "slabs", "one" if 1 << slab_log2 >= K else "several")}

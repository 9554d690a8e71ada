"""Every kernel of the 8-bit products that a call can reach, on ragged sizes, against exact sums.

The rule that chooses the kernel is evaluated on the host: every one that random sizes reach
has to be among those that the lists below reach.
"""
import ctypes
import math
import os
import random
import subprocess
import tempfile

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import check, offsets_of, padded  # noqa: E402
from .test_q8 import BF16, F32, bytes_of, positive, product  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """#include "%s/fp32_gemm_04_amd/csrc/lm_rule.hpp"
extern "C" int rule(int fast, int64_t used, int64_t rows, int64_t N, int64_t K)
{
    return sgemm::lm::byte_rows_tile(fast, used, rows, N, K, 256);
}
extern "C" int few(int fast, int64_t groups, int64_t used, int64_t rows)
{
    return sgemm::lm::byte_few_rows(fast, groups, used, rows);
}
"""
# (rows, N, K) of one group and (groups, rows, N, K), by whether the operands take direct loads.
ONE = {True: [(18, 33, 35), (2071, 67, 102), (2094, 66, 33), (16789, 34, 34), (17794, 129, 38), (16512, 650, 68),
              (300, 2060, 4100), (8170, 34, 35), (15, 10400, 34), (41, 900, 2050), (640, 1250, 547)],
       False: [(18, 33, 35), (2071, 67, 102), (2094, 66, 33), (16789, 34, 34), (300, 2060, 4099), (5, 70, 33),
               (520, 1300, 143), (3040, 2070, 199), (70, 530, 2049)]}
GROUPS = {True: [(1, 18, 33, 35), (1, 4314, 34, 94), (2, 2094, 66, 33), (19, 15982, 34, 35), (5, 22, 13207, 34),
                 (28, 4680, 2004, 70), (32, 2048, 1530, 2000), (75, 9, 70, 130), (1, 380, 2300, 650),
                 (220, 4600, 34, 35), (3, 5, 3500, 134), (6, 150, 700, 1030)],
          False: [(1, 18, 33, 35), (1, 4314, 34, 94), (2, 2094, 66, 33), (19, 15982, 34, 35), (8, 2000, 700, 1517),
                  (3, 7, 70, 130), (6, 2662, 250, 119), (1, 2790, 1420, 9), (5, 90, 530, 2049)]}


def _load():
    with tempfile.TemporaryDirectory(prefix="q8_rule_") as d:
        source, lib = os.path.join(d, "rule.cpp"), os.path.join(d, "rule.so")
        with open(source, "w") as f:
            f.write(SOURCE % ROOT)
        subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", lib, source], check=True)
        lib = ctypes.CDLL(lib)
    i, l = ctypes.c_int, ctypes.c_int64
    lib.rule.argtypes = [i, l, l, l, l]
    lib.few.argtypes = [i, l, l, l]
    return lib


def kernel(lib, fast, groups, rows, N, K):
    used = min(groups, rows) or 1
    if lib.few(fast, groups, used, rows):
        return "few rows", fast, groups > 0
    return lib.rule(fast, used if groups else 0, rows, N, K), fast, groups > 0


def test_every_tile_is_reached():
    lib, rng = _load(), random.Random(3)

    def size(low, high):
        return int(math.exp(rng.uniform(math.log(low), math.log(high))))
    for fast in (True, False):
        listed = {kernel(lib, fast, 0, *c) for c in ONE[fast]} | {kernel(lib, fast, *c) for c in GROUPS[fast]}
        for _ in range(20000):
            rows, N, K = size(1, 40000), size(1, 40000), size(1, 20000)
            for groups in (0, size(1, 300)):
                k = kernel(lib, fast, groups, rows, N, K)
                assert k in listed or k[0] == "few rows", (k, groups, rows, N, K)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fast,case", [(f, c) for f in (True, False) for c in ONE[f]])
def test_one_group(dtype, fast, case):
    rows, N, K = case
    say("q8 tiles", dtype, case)
    ld = -(-K // 4) * 4 + (0 if fast else 1)
    X, W = bytes_of((rows, ld), 1)[:, :K], bytes_of((N, ld), 2)[:, :K]
    sx, sw = positive((rows,), 3), positive((N,), 4)
    ref = product(X, sx, W, sw)
    for pad, shift in ((0, 0), (8, 0), (3, 1)):
        Y = padded(torch.zeros((rows, N), dtype=dtype, device="cuda"), pad, shift)
        base = Y._base.clone()
        sg.q8_gemm(X, sx, W, sw, Y=Y)
        check(Y, ref, ref.abs(), 3, "tile")
        Y.zero_()
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(Y._base.view(bits), base.view(bits))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fast,case", [(f, c) for f in (True, False) for c in GROUPS[f]])
def test_groups(dtype, fast, case):
    groups, rows, N, K = case
    say("q8 tiles, groups", dtype, case)
    rng = random.Random(groups)
    cuts = sorted(rng.randrange(rows + 1) for _ in range(groups - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    ends, off = offsets_of(sizes, first=1)
    ld = -(-K // 4) * 4 + (0 if fast else 1)
    X, W = bytes_of((rows + 4, ld), 1)[:, :K], bytes_of((groups, N, ld), 2)[..., :K]
    sx, sw = positive((rows + 4,), 3), positive((groups, N), 4)
    Y = sg.q8_gemm(X, sx, W, sw, off, dtype=dtype)
    assert (Y[:1] == 0).all() and (Y[-3:] == 0).all()
    for e in range(groups):
        a, b = ends[e], ends[e + 1]
        ref = product(X[a:b], sx[a:b], W[e], sw[e])
        check(Y[a:b], ref, ref.abs(), 3, "group %d" % e)

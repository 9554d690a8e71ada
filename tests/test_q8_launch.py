"""8-bit launches at the largest extents: quantisation of more rows than a launch of wide
workgroups takes at once, and products of more row tiles than a launch of the smaller tiles
takes."""
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
from .test_lm_products import check  # noqa: E402
from .test_q8 import BF16, F32, bytes_of, positive, quantize_reference  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """#include "%s/fp32_gemm_04_amd/csrc/lm_rule.hpp"
using namespace sgemm::lm;
extern "C" int64_t blocks(int64_t work, int threads) { return launch_blocks(work, threads); }
"""
TILES = """#include "%s/fp32_gemm_04_amd/csrc/lm_rule.hpp"
using namespace sgemm::lm;
// Workgroups of the chosen tile, and of the largest; -1 where none is chosen.
extern "C" int64_t chosen(int fast, int64_t used, int64_t rows, int64_t N, int64_t K)
{
    const int i = byte_rows_tile(fast, used, rows, N, K, 256);
    if (i < 0) return -1;
    const ByteTileCost &t = i < NUM_TILES ? kI8Tiles[fast][i] : kI8Splits[fast][i - NUM_TILES];
    return byte_blocks(used, rows, N, t.bm, t.bn);
}
extern "C" int64_t largest(int fast, int64_t used, int64_t rows, int64_t N)
{
    return byte_blocks(used, rows, N, byte_side(fast), byte_side(fast));
}
"""
MOST = 2 ** 31 - 1025
GEMM = dict(type=1, groups=1, rows=8, N=16, K=32, X=4096, ldx=32, x_scales=8192, W=12288, ldw=32,
            stride_w=512, w_scales=16384, Y=20480, ldy=2 ** 31 - 1, offsets=0, fill=0)
ITEMS = 1 << 32  # work items of a launch along x stay below


def _load(source):
    with tempfile.TemporaryDirectory(prefix="q8_launch_") as d:
        path, lib = os.path.join(d, "rule.cpp"), os.path.join(d, "rule.so")
        with open(path, "w") as f:
            f.write(source % ROOT)
        subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", lib, path], check=True)
        return ctypes.CDLL(lib)


def test_workgroups_of_a_launch():
    lib = _load(SOURCE)
    lib.blocks.restype, lib.blocks.argtypes = ctypes.c_int64, [ctypes.c_int64, ctypes.c_int]
    for threads in (256, 512, 1024):
        for work in (1, 1000, (1 << 22) - 1, 1 << 22, 1 << 23, (1 << 23) + 9, 1 << 24, 1 << 31, 1 << 40):
            n = lib.blocks(work, threads)
            assert 1 <= n <= work and n * threads < ITEMS
            assert n == work or (n + 1) * threads >= ITEMS


def test_a_tile_is_chosen_whose_workgroups_a_launch_takes():
    lib, rng = _load(TILES), random.Random(7)
    i, l = ctypes.c_int, ctypes.c_int64
    for fn, n in ((lib.chosen, 5), (lib.largest, 4)):
        fn.restype, fn.argtypes = l, [i] + [l] * (n - 1)

    def size(high):
        return int(math.exp(rng.uniform(0, math.log(high))))
    cases = [(used, rows, N, K) for used in (0, 1, 3, 1 << 20) for rows in ((1 << 30) - 1, 1 << 30, MOST)
             for N in (1, 64, 128) for K in (1, 4, 4096)]
    cases += [(size(rows) if rng.random() < 0.5 else 0, rows, size(MOST), size(131071))
              for rows in (size(MOST) for _ in range(20000))]
    taken = 0
    for fast in (0, 1):
        for used, rows, N, K in cases:
            n, least = lib.chosen(fast, used, rows, N, K), lib.largest(fast, used, rows, N)
            assert (n < 0) == (least >= 1 << 24) and n < 1 << 24 and (n < 0 or n >= least), (fast, used, rows, N, K)
            taken += n >= 0
    assert taken > 20000


@pytest.mark.parametrize("kw,code", [
    (dict(rows=MOST, N=MOST), -4), (dict(rows=MOST, N=513), -4), (dict(rows=MOST, N=129, ldx=33), -4),
    (dict(rows=1 << 24, groups=1 << 24, offsets=4096), -4),
])
def test_products_past_a_launch_are_refused(kw, code):
    assert sg.sgemm_q8_gemm(*dict(GEMM, **kw).values()) == code


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU device node is present")
@pytest.mark.parametrize("kw", [dict(rows=MOST, N=256), dict(rows=MOST, N=128, ldx=33), dict(N=MOST),
                                dict(rows=(1 << 24) - 1, groups=1 << 24, offsets=4096, N=200)])
def test_products_of_a_launch_reach_the_device(kw):
    assert sg.sgemm_q8_gemm(*dict(GEMM, **kw).values()) > 0  # the checks pass; HIP reports no device


@pytest.fixture
def release():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.slow
def test_quantize_of_more_rows_than_wide_workgroups(release):
    """Eight waves a row, and more rows than 2^32 work items have workgroups of them for."""
    rows, K = (1 << 23) + 21, 8200
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of free memory")
    say("quantize rows", rows, K)
    at = torch.tensor([0, 1, 4095, (1 << 23) - 2, (1 << 23) - 1, 1 << 23, rows - 2, rows - 1], device="cuda")
    X = torch.empty((rows, K), dtype=BF16, device="cuda")  # other rows go nowhere
    g = torch.Generator(device="cuda").manual_seed(1)
    X[at] = torch.randn((len(at), K), generator=g, device="cuda").to(BF16)
    place = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    place[at, 0] = torch.arange(len(at), dtype=torch.int32, device="cuda")
    Q = torch.full((len(at), K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((len(at),), -1.0, device="cuda")
    status = sg.sgemm_q8_quantize(sg.SGEMM_TYPE_BF16, rows, K, X.data_ptr(), K, 1, place.data_ptr(), len(at),
                                  Q.data_ptr(), K, s.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    ref, scale = quantize_reference(X[at])
    assert torch.equal(s, scale) and torch.equal(Q, ref)


@pytest.mark.gpu
@pytest.mark.slow
@pytest.mark.parametrize("ld", [4, 3])
@pytest.mark.parametrize("groups", [0, 2])
def test_product_of_more_rows_than_small_tiles(ld, groups, release):
    """2^24 tiles of 64 rows, the fastest for one column of rows at odd bytes, and aligned ones."""
    rows, K = (1 << 30) + 77, 3
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GB of free memory")
    say("product rows", rows, ld, groups)
    at = torch.tensor([0, 1, 2, 63, (1 << 29) + 5, (1 << 30) - 1, 1 << 30, rows - 3, rows - 2, rows - 1], device="cuda")
    X, sx = torch.zeros((rows, ld), dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    X[at] = bytes_of((len(at), ld), 1)
    sx[at] = positive((len(at),), 2)
    X = X[:, :K]
    W, sw = bytes_of((max(groups, 1), 1, K), 3), positive((max(groups, 1), 1), 4)
    begin, cut, end = 1, (1 << 29) + 1, rows - 2
    off = torch.tensor([begin, cut, end], dtype=torch.int32, device="cuda") if groups else None
    Y = sg.q8_gemm(X, sx, W, sw, off, dtype=F32) if groups else sg.q8_gemm(X, sx, W[0], sw[0], dtype=F32)
    g = (at >= cut).long() if groups else torch.zeros_like(at)
    ref = (X[at].double() * W[g, 0].double()).sum(1) * sx[at].double() * sw[g, 0].double()
    if groups:
        ref[(at < begin) | (at >= end)] = 0.0
    check(Y[at, 0], ref, ref.abs(), 3, "rows")
    Y[at] = 0.0
    assert not Y.any()

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
from .test_q8 import BF16, bytes_of, positive, quantize_reference  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """#include "%s/fp32_gemm_04_amd/csrc/lm_rule.hpp"
using namespace sgemm::lm;
extern "C" int64_t blocks(int64_t work, int threads) { return launch_blocks(work, threads); }
"""
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

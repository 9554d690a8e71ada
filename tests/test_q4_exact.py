"""4-bit products on data for which every sum is exact, so that the result is the one value:
any kernel, any order of summation, any length.

x holds whole numbers up to 4 in magnitude and the scales are 1/64, 1/32 and 1/16.  In units
of the smallest scale the kernels' partial sums, of s x (16 + q) and of s x (16 + z), are whole
and at most 8192 * 4 * 31 * 4 < 2^22.  A second form has rows with four values of 17 bits, which
take all three bf16 parts of an fp32 value: at most 4 * 2^17 * 31 < 2^24 with scales of 1.
"""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from . import q4_rule  # noqa: E402
from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, offsets_of, padded  # noqa: E402
from .test_lm_tiles import split  # noqa: E402

# (groups, rows, N, K, block); no groups: one set of weights.
SMALL = [(groups, rows, 41, K, block) for block in (32, 64, 128)
         for groups, rows in ((0, 1), (0, 9), (0, 14), (0, 26), (0, 53), (1, 9), (1, 16), (1, 32), (4, 70))
         for K in (152, 1462, 8192)]
WIDE = [(0, 3, 12949, 160, 64), (3, 21, 4170, 152, 32), (1, 5, 54832, 140, 128), (0, 16, 26144, 536, 128),
        (3, 4, 4544, 194, 64), (1, 2, 19648, 142, 32), (3, 48, 35968, 148, 128), (8, 8, 33797, 144, 64),
        (1, 8, 12736, 140, 128), (0, 1, 13124, 160, 64), (1, 2, 14976, 144, 32), (1, 8, 20583, 940, 32),
        (0, 6, 14696, 152, 128), (0, 1, 13256, 188, 64), (0, 12, 28001, 2048, 32), (8, 40, 8200, 512, 64)]


def test_every_kernel_that_is_chosen_is_tested():
    tested, reached = set(), {}
    for case in SMALL + WIDE:
        for size in (2, 4):
            tested |= q4_rule.kernels(size, *case)
    rng = random.Random(2)
    for _ in range(20000):
        K = int(math.exp(rng.uniform(math.log(2), math.log(20000)))) // 2 * 2 or 2
        case = (rng.choice([0, 0, 1, 3, 16, 64]), int(math.exp(rng.uniform(0, math.log(300)))),
                int(math.exp(rng.uniform(0, math.log(60000)))), K // 8 * 8 if rng.random() < 0.5 and K >= 8 else K,
                rng.choice([32, 64, 128]))
        for size in (2, 4):
            for key in q4_rule.kernels(size, *case):
                reached.setdefault(key, case)
            rt, nt, wn, cols, pass_, slab_log2, lds = q4_rule.plan(
                size, case[0] > 0, max(case[0], 1), *case[1:])
            # What the kernel counts on: rows and LDS within bounds, a slab a chunk for each wave.
            assert pass_ <= 16 * rt and cols == 16 * nt * wn and lds <= 160 * 1024
            assert (1 << slab_log2) >= 128 * 8 // wn
    missed = {k: v for k, v in reached.items() if k not in tested}
    assert not missed, missed


def operands(case, wide_bits=False, seed=1):
    groups, rows, N, K, block = case
    g = torch.Generator().manual_seed(seed)
    lead, G = ((groups,) if groups else ()), -(-K // block)
    Q = torch.randint(0, 256, lead + (N, K // 2), generator=g).to(torch.uint8)
    Z = torch.randint(0, 16, lead + (N, G), generator=g).to(torch.uint8)
    if wide_bits:
        X = torch.zeros(rows, K)
        for r in range(rows):
            at = torch.randperm(K, generator=g)[:4]
            X[r, at] = (torch.randint(1 << 16, 1 << 17, (len(at),), generator=g) | 1).float()
        return X, Q, torch.ones(lead + (N, G)), Z
    X = torch.randint(-4, 5, (rows, K), generator=g).float()
    return X, Q, torch.randint(0, 3, lead + (N, G), generator=g).float().exp2() / 64, Z


def product(X, Q, S, Z, K, block):
    """In 64 bits, for one set of weights."""
    q = torch.stack([Q & 15, Q >> 4], -1).flatten(-2).double()
    at = torch.arange(K, device=Q.device) // block
    z = Z.double()[:, at] if Z is not None else 8.0
    return X.double() @ ((q - z) * S.double()[:, at]).t()


def test_a_misplaced_block_shows():
    """The data tells weights apart: with the two halves of every byte of one block exchanged,
    hardly any result is the same."""
    X, Q, S, Z = operands((0, 20, 50, 4096, 32))
    wrong = Q.clone()
    wrong[:, 640:656] = (Q[:, 640:656] >> 4) | (Q[:, 640:656] << 4)
    same = product(X, Q, S, Z, 4096, 32) == product(X, wrong, S, Z, 4096, 32)
    assert same.double().mean() < 0.05


def run(case, dtype, wide_bits, zeros):
    groups, rows, N, K, block = case
    X, Q, S, Z = (t.cuda() for t in operands(case, wide_bits))
    Z = Z if zeros else None
    x, s = X.to(dtype), S.to(dtype)
    x = padded(x, 3, 1) if rows % 2 else x
    ends, off = offsets_of(split(rows, groups)) if groups else ([0, rows], None)
    Y = sg.q4_matvec(x, Q, s, Z, block=block, offsets=off)
    for e in range(max(groups, 1)):
        w = (Q[e], S[e], Z[e] if zeros else None) if groups else (Q, S, Z)
        ref = product(X[ends[e]:ends[e + 1]], *w, K, block)
        assert torch.equal(Y[ends[e]:ends[e + 1]], ref.to(dtype)), e


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", SMALL + WIDE)
def test_exact(dtype, case):
    say("q4 exact", dtype, case)
    run(case, dtype, False, True)
    run(case, dtype, False, False)


@pytest.mark.gpu
@pytest.mark.parametrize("case", SMALL + WIDE)
def test_exact_with_all_bits_of_fp32(case):
    say("q4 bits", case)
    run(case, F32, True, True)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("power", [-100, -126, -133, -137])
def test_small_values_of_fp32(block, power):
    """Down to bits of 2^-133 everything is kept, below it what the last part holds under that:
    at most 2^-133 a value, times up to 31."""
    say("q4 small", block, power)
    K = 520
    X, Q, S, Z = (t.cuda() for t in operands((0, 7, 41, K, block), True))
    X *= 2.0 ** power
    Y = sg.q4_matvec(X, Q, S, Z, block=block).double()
    lost = 0 if power >= -133 else 4 * 31 * 2.0 ** -133
    assert ((Y - product(X, Q, S, Z, K, block)).abs() <= lost).all()

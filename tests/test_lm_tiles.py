"""Every tile kernel of the language-model products that a call can reach, on ragged sizes,
with outputs of every alignment.

The lists below give sizes for each type and way of loading; on the host, the rule that
chooses the tiles is evaluated on them and on many random sizes, and every kernel that the
random sizes reach has to be among those that the lists reach.
"""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from . import lm_rule  # noqa: E402
from .gpu_helpers import say  # noqa: E402
from .test_lm_products import (BF16, F32, check, check_gradients, check_loss,  # noqa: E402
                               offsets_of, padded, rand)

# (groups, rows, N, K), (groups, rows, M, N) and (rows, vocabulary, K), by type and whether
# the operands take direct loads.
ROWS = {
    (BF16, True): [(5, 21, 75, 141), (16, 7, 3485, 33), (3, 8735, 43, 74), (8, 12120, 130, 37),
                   (38, 16424, 133, 37), (1, 2440, 6856, 640), (3, 7613, 1930, 769)],
    (BF16, False): [(5, 21, 75, 141), (32, 4, 6272, 35), (5, 8465, 33, 41), (2, 12336, 144, 54)],
    (F32, True): [(5, 21, 75, 141), (1, 4160, 33, 33), (2, 9224, 72, 55), (14, 12263, 33, 33),
                  (33, 11942, 208, 34)],
    (F32, False): [(5, 21, 75, 141), (37, 3904, 33, 52), (1, 8594, 72, 64), (1, 12744, 33, 46),
                   (16, 12664, 199, 39)],
}
SUMS = {
    (BF16, True): [(1, 200, 33, 47), (39, 200, 151, 33), (26, 200, 311, 33), (38, 200, 641, 33),
                   (39, 200, 65, 831), (11, 9086, 2662, 439)],
    (BF16, False): [(1, 200, 33, 47), (39, 200, 70, 65), (24, 200, 345, 33), (22, 200, 1110, 33)],
    (F32, True): [(1, 200, 33, 47), (38, 200, 106, 33), (40, 200, 296, 33), (35, 271, 680, 65)],
    (F32, False): [(1, 200, 33, 47), (27, 200, 72, 65), (33, 200, 33, 337), (32, 200, 776, 72)],
}
XENT = {
    (BF16, True): [(1, 33, 33), (1, 24604, 1042), (130, 33, 33), (8390, 35, 40), (554, 651, 756),
                   (65, 34768, 59), (69, 26634, 516), (65, 8920, 48), (1, 184, 2068), (34, 33, 96),
                   (1, 582, 1692), (1, 1552, 2000), (35, 200, 1977), (14080, 130, 140),
                   (216, 20416, 559), (137, 568, 1848), (2923, 33, 1642), (138, 3200, 941),
                   (1792, 9106, 1696), (68, 51304, 1203), (8587, 784, 1742), (11404, 11584, 33),
                   (15496, 8456, 268)],
    (BF16, False): [(1, 33, 33), (1, 28741, 864), (136, 33, 33), (8507, 33, 34), (536, 722, 705),
                    (72, 28337, 168), (35, 16596, 70), (1, 197, 1874), (35, 33, 35), (1, 611, 1586),
                    (34, 328, 1224), (12736, 138, 136), (142, 723, 1423), (784, 1932, 1920),
                    (11200, 11781, 33), (15882, 9698, 264)],
    (F32, True): [(1, 33, 33), (17, 9154, 49), (34, 15696, 345), (8488, 70, 64), (759, 4160, 286),
                  (386, 35, 2073), (621, 33, 2066), (2592, 33, 1215), (33, 16560, 1347),
                  (111, 15967, 1632), (3200, 20928, 33), (10746, 6272, 144)],
    (F32, False): [(1, 33, 33), (19, 8910, 44), (37, 14592, 400), (8960, 72, 64), (104, 31796, 224),
                   (432, 35, 1787), (960, 33, 1358), (1896, 33, 1652), (40, 11500, 1488),
                   (299, 5058, 1945), (10496, 6208, 33), (15800, 4144, 147)],
}
KINDS = ((lm_rule.grouped, ROWS), (lm_rule.wgrad, SUMS), (lm_rule.xent, XENT))


def size_of(dtype):
    return 2 if dtype == BF16 else 4


def cases(lists):
    return [(dtype, fast, case) for (dtype, fast), at in lists.items() for case in at]


def test_every_tile_that_is_chosen_is_tested():
    tested = set()
    for rule, lists in KINDS:
        for dtype, fast, case in cases(lists):
            tested |= rule(size_of(dtype), fast, *case)
    rng = random.Random(1)

    def size(most):
        n, by = int(math.exp(rng.uniform(0, math.log(most)))), rng.choice([1, 1, 8, 64, 256])
        return n // by * by if n >= by else n

    missed = {}
    for _ in range(20000):
        drawn = [(size(64), size(20000), size(20000), size(4096)),
                 (size(64), size(20000), size(8192), size(20000)),
                 (size(16384), size(131072), size(4096))]
        for (rule, _), case in zip(KINDS, drawn):
            for bytes_ in (2, 4):
                for fast in (True, False):
                    for key in rule(bytes_, fast, *case) - tested:
                        missed.setdefault(key, case)
    assert not missed, missed


# ------------------------------------------------------------------- on the GPU

def laid_out(t, fast):
    """Rows that direct loads take, at 4-byte addresses and no better, or that they do not."""
    if t.dtype == BF16:
        return padded(t, t.shape[-1] % 2 + 2, 2) if fast else padded(t, 3, 1)
    if fast:
        return padded(t, 1, 1)
    ld = (1 << 20) + 3  # rows further apart than 2^22 bytes
    buf = torch.empty(t.shape[0] * ld, device="cuda")
    v = buf.view(t.shape[0], ld)[:, :t.shape[1]]
    v.copy_(t)
    return v


def empty(shape, dtype, pad, shift):
    return padded(torch.zeros(shape, dtype=dtype, device="cuda"), pad, shift)


def by_fours(columns):
    """Padding that makes rows of whole fours, but not of eights."""
    return -columns % 8 + 4


def same_bits(a, b):
    i = torch.int16 if a.dtype == BF16 else torch.int32
    return torch.equal(a.contiguous().view(i), b.contiguous().view(i))


@pytest.fixture(autouse=True)
def release():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def split(rows, groups):
    """Row counts that add up to rows, one of them 0 where there are more than two."""
    rng = random.Random(rows)
    cuts = sorted(rng.randrange(rows + 1) for _ in range(groups - 1))
    if groups > 2:
        cuts[1] = cuts[0]
    return [b - a for a, b in zip([0] + cuts, cuts + [rows])]


@pytest.mark.gpu
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,fast,case", cases(ROWS))
def test_rows(dtype, fast, case, trans):
    say("tiles, rows", dtype, fast, case, trans)
    E, rows, N, K = case
    ends, off = offsets_of(split(rows, E))
    X, W = rand((rows, K), dtype, 1), rand((E, N, K) if trans else (E, K, N), dtype, 2)
    x, w = laid_out(X, fast), laid_out(W, True) if dtype == F32 else laid_out(W, fast)
    Y = sg.grouped_gemm(x, w, off, trans=trans)
    old = rand((rows, N), dtype, 3)
    scaled = padded(old, 1 + N % 2, 1)
    sg.grouped_gemm(x, w, off, scaled, trans=trans, alpha=-0.5, beta=2.0)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        u, v = X[a:b].double(), (W[e].t() if trans else W[e]).double()
        ref, mag, before = u @ v, u.abs() @ v.abs(), old[a:b].double()
        check(Y[a:b], ref, mag, K + 2, "rows of %d" % e)
        check(scaled[a:b], 2 * before - 0.5 * ref, 2 * before.abs() + 0.5 * mag, K + 4, "scaled")
    for pad, shift in ((by_fours(N), 4), (N % 2 + 1, 1)):
        out = empty((rows, N), dtype, pad, shift)
        outside = out._base.isnan().sum()
        sg.grouped_gemm(x, w, off, out, trans=trans)
        assert same_bits(out, Y) and out._base.isnan().sum() == outside


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fast,case", cases(SUMS))
def test_sums(dtype, fast, case):
    say("tiles, sums", dtype, fast, case)
    E, rows, M, N = case
    ends, off = offsets_of(split(rows, E))
    X, G = rand((rows, M), dtype, 1), rand((rows, N), dtype, 2)
    x, g = laid_out(X, fast), laid_out(G, True) if dtype == F32 else laid_out(G, fast)
    D = sg.grouped_wgrad(x, g, off)
    old = rand((E, M, N), dtype, 3)
    scaled = padded(old, 1 + N % 2, 1)
    sg.grouped_wgrad(x, g, off, scaled, alpha=1.5, beta=-1.0)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        u, v = X[a:b].double().t(), G[a:b].double()
        ref, mag, before = u @ v, u.abs() @ v.abs(), old[e].double()
        check(D[e], ref, mag, b - a + 2, "sums of %d" % e)
        check(scaled[e], 1.5 * ref - before, 1.5 * mag + before.abs(), b - a + 4, "scaled")
    for pad, shift in ((by_fours(N), 4), (N % 2 + 1, 1)):
        out = empty((E, M, N), dtype, pad, shift)
        outside = out._base.isnan().sum()
        sg.grouped_wgrad(x, g, off, out)
        assert same_bits(out, D) and out._base.isnan().sum() == outside


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fast,case", cases(XENT))
def test_losses(dtype, fast, case):
    say("tiles, losses", dtype, fast, case)
    T, V, K = case
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 2.0 / K ** 0.5)
    x, w = laid_out(X, fast), laid_out(W, fast)
    g = torch.Generator().manual_seed(3)
    targets = torch.randint(0, V, (T,), generator=g)
    targets[3::7] = -100
    targets[5::11] = V
    targets[0] = V - 1
    targets, dloss = targets.cuda(), (torch.rand(T, generator=g) + 0.5).cuda() / T
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    check_loss(X, W, targets, loss, lse)
    dX, dW = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    # Up to 128 bf16 rows keep 16 bits of each derivative.
    check_gradients(X, W, targets, dloss, dX, dW, half_d=2.0 ** -16 if dtype == BF16 and T <= 128 else None)
    for pad, shift in ((by_fours(K), 4), (K % 2 + 1, 1)):
        outs = [empty(t.shape, dtype, pad, shift) for t in (dX, dW)]
        outside = [t._base.isnan().sum() for t in outs]
        sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, *outs)
        assert same_bits(outs[0], dX) and same_bits(outs[1], dW)
        assert [t._base.isnan().sum() for t in outs] == outside

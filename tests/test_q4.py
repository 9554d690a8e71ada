"""Products with weights held in 4 bits, and their quantisation, on the GPU,
against their definitions in float64."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, check, offsets_of, padded, rand  # noqa: E402

pytestmark = pytest.mark.gpu


def weights(shape, K, block, dtype, seed, zeros=True):
    g = torch.Generator().manual_seed(seed)
    G = -(-K // block)
    Q = torch.randint(0, 256, shape + (K // 2,), generator=g).to(torch.uint8).cuda()
    S = (torch.rand(shape + (G,), generator=g) + 0.5).to(dtype).cuda()
    Z = torch.randint(0, 16, shape + (G,), generator=g).to(torch.uint8).cuda() if zeros else None
    return Q, S, Z


def dequantised(Q, S, Z, K, block):
    """(w, (16 + q) s): the weights and the magnitudes the sums pass through."""
    q = torch.stack([Q & 15, Q >> 4], -1).flatten(-2).double()
    at = torch.arange(K, device="cuda") // block
    s = S.double()[..., at]
    z = Z.double()[..., at] if Z is not None else 8.0
    return (q - z) * s, (16 + q) * s.abs()


def check_rows(Y, X, Q, S, Z, K, block, what):
    """A block's sums of x (16 + q) and of x, times up to 31: K products in all, each
    addition within 2^-24 of a partial sum that sum |x| (16 + q) bounds (sum |x| times
    (16 + z) is at most twice that), and the joins of blocks, waves and parts."""
    w, m = dequantised(Q, S, Z, K, block)
    check(Y, X.double() @ w.t(), X.double().abs() @ m.t(), 4 * (K + 16), what)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 2), (1, 17, 34), (1, 64, 128), (2, 100, 1000), (5, 48, 4096),
                                      (6, 33, 514), (16, 40, 256), (17, 40, 320), (40, 24, 2050),
                                      (70, 130, 96), (3, 8200, 288)])
def test_q4_matvec(dtype, block, rows, N, K):
    say("q4", dtype, block, rows, N, K)
    X = rand((rows, K), dtype, 1)
    for zeros in (True, False):
        Q, S, Z = weights((N,), K, block, dtype, 2, zeros)
        Y = sg.q4_matvec(X, Q, S, Z, block=block)
        check_rows(Y, X, Q, S, Z, K, block, "q4")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block", [32, 128])
def test_q4_groups(dtype, block):
    """One set of weights per group; padded rows; rows of no group left alone."""
    ends, off = offsets_of([1, 0, 20, 3, 70], first=2)
    rows, N, K = ends[-1] + 3, 50, 352
    X = padded(rand((rows, K), dtype, 1), 3)
    Q, S, Z = weights((5, N), K, block, dtype, 2)
    Y0 = rand((rows, N), dtype, 3)
    Y = padded(Y0, 5)
    sg.q4_matvec(X, Q, S, Z, block=block, Y=Y, offsets=off)
    for e in range(5):
        a, b = ends[e], ends[e + 1]
        check_rows(Y[a:b], X[a:b], Q[e], S[e], Z[e], K, block, "group %d" % e)
    assert torch.equal(Y[:2], Y0[:2]) and torch.equal(Y[ends[-1]:], Y0[ends[-1]:])


def test_q4_fp32_rows_keep_their_bits():
    """x = 1 + 2^-23 times a single weight of 1 comes back whole, also next to
    values far larger in other blocks' rows."""
    K, N = 256, 16
    X = torch.zeros((3, K), device="cuda")
    X[0, 5], X[1, 200], X[2, 7] = 1 + 2.0 ** -23, -(1 + 2.0 ** -23) * 2.0 ** -40, 2.0 ** 90
    Q = torch.full((N, K // 2), 0x99, dtype=torch.uint8, device="cuda")  # 9 - 8 = 1
    S = torch.ones((N, 2), device="cuda")
    Y = sg.q4_matvec(X, Q, S)
    for r, k in ((0, 5), (1, 200), (2, 7)):
        v = X[r, k].double()
        assert ((Y[r].double() - v).abs() <= 26 * 2.0 ** -23 * v.abs()).all()
    one = sg.q4_matvec(X[:1], Q, S)
    assert torch.equal(one[0], Y[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_q4_empty(dtype):
    Q, S, Z = weights((7,), 64, 32, dtype, 1)
    assert sg.q4_matvec(rand((0, 64), dtype, 1), Q, S, Z, block=32).shape == (0, 7)
    Y = sg.q4_matvec(rand((3, 0), dtype, 1), Q[:, :0], S[:, :0].contiguous(), block=32)
    assert not Y.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("N,K", [(1, 2), (5, 130), (33, 1024)])
def test_q4_quantize(dtype, block, zeros, N, K):
    W = padded(rand((N, K), dtype, 1), 6)
    W[0, :2] = 0
    Q, S, Z = sg.q4_quantize(W, block, zeros)
    G = -(-K // block)
    full = torch.zeros((N, G * block), device="cuda")
    full[:, :K] = W.float()
    v = full.view(N, G, block)
    lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
    # Divided in 64 bits, which rounds to fp32 as one fp32 division does (torch's fp32
    # division by a number multiplies by its reciprocal).
    scale = (hi - lo).double() / 15 if zeros else torch.maximum(hi, -lo).double() / 7
    scale = scale.float().to(dtype)
    assert torch.equal(S, scale)
    s = scale.float()
    z = ((-lo / s).round().clamp(0, 15) if zeros else torch.full_like(s, 8)).nan_to_num(0)
    q = ((v / s[..., None]).round() + z[..., None]).clamp(0, 15)
    q = torch.where(s[..., None] > 0, q, z[..., None]).flatten(1)[:, :K].to(torch.uint8)
    assert torch.equal(torch.stack([Q & 15, Q >> 4], -1).flatten(-2), q)
    assert (Z is None) if not zeros else torch.equal(Z, z.to(torch.uint8))
    # Every weight reads back within half a scale (and what rounding the scale to the
    # type and clamping can add: 15 steps of 2^-8 of it, and the zero's own half step).
    w, _ = dequantised(Q, S, Z, K, block)
    at = torch.arange(K, device="cuda") // block
    assert ((w - W.double()).abs() <= (1.0 + 15 * 2.0 ** -8) * s.double()[:, at] + 1e-30).all()

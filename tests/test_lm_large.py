"""Cross entropy and 4-bit products on operands past 2^31 elements or bytes, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, padded, rand  # noqa: E402
from .test_q4_exact import product  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


@pytest.fixture(autouse=True)
def release():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def close(out, ref, mag, what):
    """Sums of d x or d w: each d, exact but for 2^-16 (bf16's two parts) and the exponential's
    argument and value, 2^-18 at |z - lse| < 32, and fp32 sums of at most 2^21 terms of like
    size, 2^-16 in a chain of 256 partial sums; bf16 results are rounded by 2^-8."""
    half = 2.0 ** -8 if out.dtype == BF16 else 0.0
    bad = ~((out.double() - ref).abs() <= 2.0 ** -14 * mag + half * ref.abs() + 1e-37)
    assert not bad.any(), "%s: %d of %d" % (what, int(bad.sum()), bad.numel())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_vocabulary_past_32_bits(dtype):
    T, K, V = 3, 2048, (1 << 20) + 5003
    assert V * K > 1 << 31
    say("vocabulary past 2^31 values", dtype)
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 2.0 / K ** 0.5)
    targets = torch.tensor([V - 1, 7, 1 << 20], device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    z = torch.cat([X.double() @ w.double().t() for w in W.split(1 << 17)], 1)
    ref = torch.logsumexp(z, 1)
    # Logits within (K + 1) 2^-24 sum|x w|; the sum is near 0.64 * 2 sqrt(K) = 58: 0.0071.
    assert ((lse.double() - ref).abs() < 0.01).all()
    assert ((loss.double() - (ref - z.gather(1, targets[:, None])[:, 0])).abs() < 0.02).all()
    dloss = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    # d from the kernels' own lse, whose error every d of the row shares.
    d = (z - lse.double()[:, None]).exp()
    d[torch.arange(T), targets] -= 1
    d *= dloss.double()[:, None]
    ref, mag = 0, 0
    for a, w in zip(range(0, V, 1 << 17), W.split(1 << 17)):
        c = d[:, a:a + (1 << 17)]
        ref, mag = ref + c @ w.double(), mag + c.abs() @ w.double().abs()
        if a % (1 << 19) == 0 or a + (1 << 17) >= V:
            close(dW[a:a + 4000], c[:, :4000].t() @ X.double(), c[:, :4000].t().abs() @ X.double().abs(), "dW")
    close(dW[-4000:], d[:, -4000:].t() @ X.double(), d[:, -4000:].t().abs() @ X.double().abs(), "dW")
    close(dX, ref, mag, "dX")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_past_32_bits(dtype):
    T, K, V = (1 << 20) + 3001, 2048, 40
    assert T * K > 1 << 31
    say("rows past 2^31 values", dtype)
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 2.0 / K ** 0.5)
    targets = torch.randint(0, V, (T,), device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    tail = slice(T - 2000, T)
    short, _ = sg.linear_cross_entropy(X[tail], W, targets[tail])
    z = X[tail].double() @ W.double().t()
    ref = torch.logsumexp(z, 1)
    assert ((lse[tail].double() - ref).abs() < 0.01).all()
    assert ((loss[tail].double() - (ref - z.gather(1, targets[tail, None])[:, 0])).abs() < 0.02).all()
    assert ((loss[tail] - short).abs() < 0.04).all()
    dloss = torch.rand(T, device="cuda") + 0.5
    dX, _ = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse, need_dW=False)
    d = (z - lse[tail].double()[:, None]).exp()
    d[torch.arange(2000), targets[tail]] -= 1
    d *= dloss[tail].double()[:, None]
    # With so many rows each bf16 derivative is rounded, by 2^-8 of itself.
    mag = d.abs() @ W.double().abs()
    close(dX[tail], d @ W.double(), mag * (1 if dtype == F32 else 2 ** 7), "dX")


def exact_weights(shape, K, block, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    G = -(-K // block)
    Q = torch.randint(0, 256, shape + (K // 2,), generator=g, device="cuda", dtype=torch.uint8)
    S = torch.randint(0, 3, shape + (G,), generator=g, device="cuda").to(dtype).exp2()
    return Q, S, torch.randint(0, 16, shape + (G,), generator=g, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,rows", [(4096, 1), (4098, 5)])
def test_4_bit_columns_past_32_bits(dtype, K, rows):
    N = (1 << 20) + 4007
    assert N * (K // 2) > 1 << 31
    say("4-bit columns past 2^31 bytes", dtype, K, rows)
    Q, S, Z = exact_weights((N,), K, 128, dtype)
    X = torch.randint(-4, 5, (rows, K), device="cuda").to(dtype)
    Y = sg.q4_matvec(X, Q, S, Z)
    for a in (0, N // 2, (1 << 20) - 1000, N - 4000):
        at = slice(a, a + 4000)
        assert torch.equal(Y[:, at], product(X, Q[at], S[at], Z[at], K, 128).to(dtype)), a


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_4_bit_groups_past_32_bits(dtype):
    E, N, K = 67, 8192, 8192
    assert E * N * (K // 2) > 1 << 31
    say("4-bit groups past 2^31 bytes", dtype)
    Q, S, Z = exact_weights((E, N), K, 64, dtype)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1:] = 3
    X = torch.randint(-4, 5, (3, K), device="cuda").to(dtype)
    Y = sg.q4_matvec(X, Q, S, Z, block=64, offsets=off)
    assert torch.equal(Y, product(X, Q[-1], S[-1], Z[-1], K, 64).to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_4_bit_rows_far_apart(dtype):
    """Rows of X and of Y that lie 2^30 elements apart."""
    say("rows far apart", dtype)
    Q, S, Z = exact_weights((50,), 512, 32, dtype)
    ld, rows = (1 << 30) + 8, 5
    X = torch.empty(rows * ld, dtype=dtype, device="cuda").view(rows, ld)[:, :512]
    X.copy_(torch.randint(-4, 5, (rows, 512), device="cuda"))
    Y = torch.empty(rows * ld, dtype=dtype, device="cuda").view(rows, ld)[:, :50]
    sg.q4_matvec(X, Q, S, Z, block=32, Y=Y)
    assert torch.equal(Y, product(X, Q, S, Z, 512, 32).to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantised_weights_past_32_bits(dtype):
    N, K = (1 << 20) + 3001, 2050
    assert N * K > 1 << 31
    say("quantised weights past 2^31 values", dtype)
    W = rand((N, K), dtype, 1)
    Q, S, Z = sg.q4_quantize(W, 64)
    for a in (0, (1 << 20) - 500, N - 1000):
        for whole, part in zip((Q, S, Z), sg.q4_quantize(padded(W[a:a + 1000], 2), 64)):
            assert torch.equal(whole[a:a + 1000], part), a

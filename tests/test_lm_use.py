"""The language-model products as a program uses them, on the GPU: the layers
of a model together, captured graphs, streams, and sizes past the small tests'.
"""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import (BF16, F32, check, check_gradients, check_loss,  # noqa: E402
                               grouped_reference, offsets_of, padded, rand)
from .test_q4 import check_rows, weights  # noqa: E402

pytestmark = pytest.mark.gpu

# Every tile: (rows of each group, N, K), from a few rows to the largest tile's.
TILED = [([40] * 5, 260, 200), ([150, 0, 97], 700, 328), ([600, 513], 1000, 264),
         ([1300, 900, 40], 2100, 136), ([4200, 4000], 2048, 96)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,N,K", TILED)
def test_grouped_every_tile(dtype, trans, sizes, N, K):
    say("grouped tiles", dtype, trans, sizes, N, K)
    ends, off = offsets_of(sizes)
    X, E = rand((ends[-1], K), dtype, 1), len(sizes)
    W = rand((E, N, K) if trans else (E, K, N), dtype, 2)
    Y = sg.grouped_gemm(X, W, off, trans=trans)
    ref, mag = grouped_reference(X, W, ends, trans, 1.0, 0.0, torch.zeros_like(Y))
    check(Y, ref, mag, K + 2, "grouped")
    G = rand((ends[-1], N), dtype, 3)
    D = sg.grouped_wgrad(G, X, off) if trans else sg.grouped_wgrad(X, G, off)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        x, g = X[a:b].double(), G[a:b].double()
        x, g = (g.t(), x) if trans else (x.t(), g)
        check(D[e], x @ g, x.abs() @ g.abs(), b - a + 2, "wgrad")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,V", [(600, 200, 5000), (2100, 136, 9000), (4096, 64, 16500), (700, 513, 4001)])
def test_xent_every_tile(dtype, T, K, V):
    """Larger tiles, several pieces' worth of columns in one, and slices of dX's sum."""
    say("xent tiles", dtype, T, K, V)
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 2.0 / K ** 0.5)
    g = torch.Generator().manual_seed(3)
    targets = torch.randint(0, V, (T,), generator=g)
    targets[::9] = -1
    targets = targets.cuda()
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    check_loss(X, W, targets, loss, lse)
    dloss = torch.rand(T, generator=g).cuda() / T
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    check_gradients(X, W, targets, dloss, dX, dW)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_xent_in_several_pieces(dtype):
    """More than 256 MiB of derivatives: the vocabulary goes in pieces, and dX sums over them."""
    T, K, V = 33000, 16, 4500
    assert T * V * (4 if dtype == F32 else 2) > 1 << 28
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 0.5)
    targets = torch.randint(0, V, (T,), device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    at = torch.arange(0, T, 331, device="cuda")  # rows of dX stand alone
    check_loss(X[at], W, targets[at], loss[at], lse[at])
    check_gradients(X[at], W, targets[at], dloss[at], dX[at], None)
    # All of dW, on a sample of its rows' inputs at a time: its sum is over every row.
    ref, mag = torch.zeros(V, K, dtype=torch.float64, device="cuda"), torch.zeros(V, K, device="cuda").double()
    for a in range(0, T, 3300):
        z = X[a:a + 3300].double() @ W.double().t()
        d = (z - torch.logsumexp(z, 1, keepdim=True)).exp()
        d[torch.arange(len(z), device="cuda"), targets[a:a + 3300]] -= 1
        d /= T
        ref += d.t() @ X[a:a + 3300].double()
        mag += d.t().abs() @ X[a:a + 3300].double().abs()
    # d: 2^-8 (bf16) of itself, the fp32 exponent's argument and value 2^-20 at |z - lse| < 12.
    off = (2.0 ** -8 if dtype == BF16 else 0.0) + 2.0 ** -20
    check(dW, ref, mag, (off * 2.0 ** 24) + T + 2, "dW")


@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 31, 33, 64, 65, 128, 129])
@pytest.mark.parametrize("K", [64, 75])
def test_xent_few_rows_keep_their_derivatives(T, K):
    """bf16 with up to 128 rows: each derivative keeps 16 bits (its rounding, 2^-8 of itself,
    and that of the remainder, 2^-8 of at most that), so that the gradients are those of
    unrounded derivatives rounded once; from 129 rows on, each derivative is rounded."""
    V = 700
    X, W = rand((T, K), BF16, 1), rand((V, K), BF16, 2, 2.0 / K ** 0.5)
    targets = torch.randint(0, V, (T,), device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    dloss = torch.rand(T, device="cuda") + 0.1
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    check_gradients(X, W, targets, dloss, dX, dW, half_d=2.0 ** -16 if T <= 128 else 2.0 ** -8)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_xent_strides_and_outside(dtype):
    """Padded and misaligned rows; only the gradients' own windows are written."""
    T, K, V = 70, 45, 333
    X, W = padded(rand((T, K), dtype, 1), 5, 1), padded(rand((V, K), dtype, 2, 0.3), 3, 1)
    targets = torch.randint(0, V, (T,), device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    check_loss(X, W, targets, loss, lse)
    dX, dW = padded(rand((T, K), dtype, 3), 7, 1), padded(rand((V, K), dtype, 4), 2, 1)
    outside = [t._base.isnan().sum() for t in (dX, dW)]
    dloss = torch.rand(T, device="cuda")
    sg.linear_cross_entropy_backward(dloss, X, W, targets, lse, dX=dX, dW=dW)
    assert [t._base.isnan().sum() for t in (dX, dW)] == outside
    check_gradients(X, W, targets, dloss, dX, dW)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_xent_rows_that_do_not_count(dtype):
    """A row of NaN or infinities that does not count leaves the gradients clean; without any
    row that counts they are zero, and with no row at all dW is."""
    T, K, V = 40, 64, 500
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 0.3)
    X[3], X[17, 5] = float("nan"), float("inf")
    targets = torch.randint(0, V, (T,), device="cuda")
    targets[3] = targets[17] = -100
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    assert loss[3] == 0 and loss[17] == 0 and not loss.isnan().any() and lse[3].isnan()
    dloss = torch.ones(T, device="cuda")
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    assert not dX[3].any() and not dX[17].any() and not dX.isnan().any()
    counts = targets >= 0
    check_gradients(X[counts], W, targets[counts], dloss[counts], dX[counts], None)
    X[3], X[17, 5] = 0, 0
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, torch.full_like(targets, V), lse)
    assert not dX.any() and not dW.any()
    loss, lse = sg.linear_cross_entropy(X[:0], W, targets[:0])
    dW.fill_(1)
    dX, dW = sg.linear_cross_entropy_backward(loss, X[:0], W, targets[:0], lse, dW=dW)
    assert dX.shape == (0, K) and not dW.any()


def test_xent_large_logits():
    """Logits of thousands: the running maximum keeps the sums in range."""
    X, W = rand((20, 64), F32, 1, 30.0), rand((3000, 64), F32, 2, 10.0)
    targets = torch.randint(0, 3000, (20,), device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    check_loss(X, W, targets, loss, lse)
    assert loss.isfinite().all()


def test_xent_gradient_against_differences():
    """The loss's own change along random directions, in the kernel's arithmetic: the
    directional derivative by central differences at step h is off by h^2/6 of the third
    derivative and by the loss's rounding over h."""
    T, K, V = 24, 32, 200
    X, W = rand((T, K), F32, 1, 0.5), rand((V, K), F32, 2, 0.3)
    targets = torch.randint(0, V, (T,), device="cuda")
    dloss = torch.ones(T, device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    U, Z = rand((T, K), F32, 3), rand((V, K), F32, 4)
    h = 2.0 ** -7
    for D, G, at in ((U, dX, 0), (Z, dW, 1)):
        args = lambda s: (X + s * D, W) if at == 0 else (X, W + s * D)  # noqa: E731
        up, down = (sg.linear_cross_entropy(*args(s), targets)[0].double().sum() for s in (h, -h))
        slope = float((G.double() * D.double()).sum())
        # Rounding: T losses near log V, each within 2^-18; third derivative: at most
        # 6 T |step|^3 of logits that move by at most 20 a unit step.
        z = (D.double() @ W.double().t()) if at == 0 else (X.double() @ D.double().t())
        bound = T * 2.0 ** -18 / h + h * h * T * float(z.abs().amax()) ** 3
        assert abs(float(up - down) / (2 * h) - slope) <= bound


def model(dtype, T=48, H=96, F=160, V=500, E=4):
    sizes = [11, 0, 30, 7]
    ends, off = offsets_of(sizes)
    X = rand((T, H), dtype, 1)
    A, B = rand((E, H, F), dtype, 2, H ** -0.5), rand((E, H, F), dtype, 3, F ** -0.5)
    O = rand((V, H), dtype, 4, H ** -0.5)
    g = torch.Generator().manual_seed(5)
    targets = torch.randint(0, V, (T,), generator=g).cuda()
    return X, A, B, O, off, ends, targets


def step(X, A, B, O, off, targets, dloss):
    """Two expert layers and the output layer's loss, and every gradient."""
    Hid = sg.grouped_gemm(X, A, off)
    Y = sg.grouped_gemm(Hid, B, off, trans=True)
    loss, lse = sg.linear_cross_entropy(Y, O, targets)
    dY, dO = sg.linear_cross_entropy_backward(dloss, Y, O, targets, lse)
    dHid = sg.grouped_gemm(dY, B, off)
    dB = sg.grouped_wgrad(dY, Hid, off)
    dX = sg.grouped_gemm(dHid, A, off, trans=True)
    dA = sg.grouped_wgrad(X, dHid, off)
    return loss, dX, dA, dB, dO


def test_layers_together():
    """Experts, output layer and loss in fp32 against autograd in float64.  Each gradient
    passes five products of at most 500 terms: within 6 * 500 * 2^-24 = 2^-12.4 of the
    magnitudes it sums over, which stay below ten times the largest gradient here."""
    X, A, B, O, off, ends, targets = model(F32)
    dloss = torch.full((len(X),), 1.0 / len(X), device="cuda")
    got = step(X, A, B, O, off, targets, dloss)
    leaves = [t.double().requires_grad_() for t in (X, A, B, O)]
    x, a, b, o = leaves
    rows = [(x[s:t] @ a[e]) @ b[e].t() for e, (s, t) in enumerate(zip(ends, ends[1:]))]
    loss = torch.nn.functional.cross_entropy(torch.cat(rows) @ o.t(), targets, reduction="none")
    grads = torch.autograd.grad(loss.mean(), leaves)
    assert (got[0].double() - loss).abs().max() <= 500 * 2.0 ** -24 * 64
    for out, ref in zip(got[1:], grads):
        assert (out.double() - ref).abs().max() <= 10 * 2.0 ** -12.4 * ref.abs().max()


def test_output_layer_in_4_bits():
    """The trained output layer quantised and used for single tokens, experts' too."""
    X, A, B, O, off, ends, targets = model(BF16, H=128, F=128)
    for block in (32, 128):
        Q, S, Z = sg.q4_quantize(O, block)
        for r in (1, 5):
            check_rows(sg.q4_matvec(X[:r], Q, S, Z, block=block), X[:r], Q, S, Z, 128, block, "tokens")
        W = B.transpose(1, 2).contiguous()  # (groups, N, K)
        Q, S, Z = sg.q4_quantize(W, block)
        Y = sg.q4_matvec(X, Q, S, Z, block=block, offsets=off)
        for e in range(4):
            a, b = ends[e], ends[e + 1]
            check_rows(Y[a:b], X[a:b], Q[e], S[e], Z[e], 128, block, "experts")


def bits(ts):
    return [t.clone().view(torch.int16 if t.dtype == BF16 else torch.int32) for t in ts]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graphs(dtype):
    """A captured training step and a captured 4-bit product: replays on new inputs, with
    eager work between them, give the eager bits; two graphs keep workspaces apart."""
    X, A, B, O, off, ends, targets = model(dtype)
    dloss = torch.full((len(X),), 1.0 / len(X), device="cuda")
    Q, S, Z = weights((4, 160), 96, 32, dtype, 7)
    run = lambda: step(X, A, B, O, off, targets, dloss) + (  # noqa: E731
        sg.q4_matvec(X, Q, S, Z, block=32, offsets=off),)
    run()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for k in range(4):
        X.copy_(rand(X.shape, dtype, 20 + k))
        targets.copy_(torch.randint(0, len(O), targets.shape, device="cuda"))
        want = bits(run())
        for g in graphs:
            g.replay()
        run()
        torch.cuda.synchronize()
        for o in outs:
            for got, ref in zip(bits(o), want):
                assert torch.equal(got, ref)


def test_streams():
    """A side stream, by argument and as the current one; results and what is allocated there
    are that stream's; the same bits as on the main stream; a stream of streams at once."""
    X, A, B, O, off, ends, targets = model(BF16, T=48)
    dloss = torch.full((len(X),), 1.0 / len(X), device="cuda")
    want = bits(step(X, A, B, O, off, targets, dloss))
    Y = sg.grouped_gemm(X, A, off)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(step(X, A, B, O, off, targets, dloss))
    side = [sg.grouped_gemm(X, A, off, stream=s) for s in streams]
    loss = sg.linear_cross_entropy(X, O, targets, stream=streams[0])[0]
    torch.cuda.synchronize()
    for o in outs:
        for got, ref in zip(bits(o), want):
            assert torch.equal(got, ref)
    for t in side:
        assert torch.equal(t, Y)
    assert torch.equal(loss, sg.linear_cross_entropy(X, O, targets)[0])


def test_results_repeat():
    """No result depends on timing: the same bits every time."""
    X, A, B, O, off, ends, targets = model(F32)
    dloss = torch.rand(len(X), device="cuda")
    first = bits(step(X, A, B, O, off, targets, dloss))
    for _ in range(3):
        for got, ref in zip(bits(step(X, A, B, O, off, targets, dloss)), first):
            assert torch.equal(got, ref)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Rows and weights that lie more than 2^32 bytes, and 2^31 elements, into their tensors."""
    K, N, rows = 64, 64, (1 << 25) + 700
    assert rows * K > 1 << 31
    X = torch.zeros((rows, K), dtype=BF16, device="cuda")
    X[-700:] = rand((700, K), BF16, 1)
    W = rand((2, N, K), BF16, 2)
    off = torch.tensor([0, 10, rows], dtype=torch.int32, device="cuda")
    Y = sg.grouped_gemm(X, W, off, trans=True)
    tail, w = X[-700:].double(), W[1].double().t()
    check(Y[-700:], tail @ w, tail.abs() @ w.abs(), K + 2, "rows")
    assert not Y[:-700].any()
    D = sg.grouped_wgrad(Y, X, off)
    y = Y[-700:].double().t()
    check(D[1], y @ tail, y.abs() @ tail.abs(), 702, "wgrad")  # zeros add nothing, and exactly
    assert not D[0].any()
    del X, Y, D
    E, N, K = 70, 8192, 4096  # 70 * 8192 * 4096 weights: 4.7 GB of bf16
    W = torch.zeros((E, N, K), dtype=BF16, device="cuda")
    W[-1] = rand((N, K), BF16, 3)
    X = rand((5, K), BF16, 4)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 5
    Y = sg.grouped_gemm(X, W, off, trans=True)
    x, w = X.double(), W[-1].double().t()
    check(Y, x @ w, x.abs() @ w.abs(), K + 2, "weights")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_empty_contraction_is_zero_whatever_alpha(dtype):
    say("empty contraction", dtype)
    off = torch.tensor([0, 3, 3], dtype=torch.int32, device="cuda")
    inf = float("inf")
    Y = sg.grouped_gemm(rand((3, 0), dtype, 1), rand((2, 0, 7), dtype, 2), off,
                        torch.ones((3, 7), dtype=dtype, device="cuda"), alpha=inf, beta=2.0)
    assert torch.equal(Y, torch.full_like(Y, 2.0))
    D = sg.grouped_wgrad(rand((3, 5), dtype, 3), rand((3, 7), dtype, 4), off, alpha=inf)
    assert torch.equal(D[1], torch.zeros_like(D[1]))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wgrad_groups_side_by_side(dtype):
    """D_e in the columns of one matrix with rows of all groups."""
    say("side by side", dtype)
    ends, off = offsets_of([70, 0, 33])
    X, G = rand((ends[-1], 50), dtype, 1), rand((ends[-1], 24), dtype, 2)
    D = torch.full((50, 3, 24), 9.0, dtype=dtype, device="cuda")
    sg.grouped_wgrad(X, G, off, D.permute(1, 0, 2))
    assert torch.equal(D.permute(1, 0, 2), sg.grouped_wgrad(X, G, off))
    with pytest.raises(sg.SgemmError, match="parameter 14"):
        sg.grouped_wgrad(X, G, off, D[:, :1].permute(1, 0, 2).expand(3, 50, 24))


def test_more_than_2_to_32_work_items():
    say("many blocks to quantise")
    n = (1 << 28) + 37
    W = torch.tensor([3.0, -1.0], dtype=BF16, device="cuda").repeat(n, 1)
    W[-1] = torch.tensor([7.0, 0.5], dtype=BF16, device="cuda")
    Q, S, _ = sg.q4_quantize(W, 32, zeros=False)
    assert Q[-1, 0].item() == 15 + 16 * 8 and S[-1].item() == 1.0  # 0.5 rounds to even
    assert torch.equal(Q[:-1], Q[:1].expand(n - 1, 1)) and torch.equal(S[:-1], S[:1].expand(n - 1, 1))
    del W, Q, S
    say("many rows of a loss")
    n = (1 << 26) + 5
    X = torch.full((n, 1), 2.0, device="cuda")
    X[-1] = -1.0
    W = torch.tensor([[1.0], [0.0]], device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, torch.zeros(n, dtype=torch.int64, device="cuda"))
    one = torch.log(torch.exp(torch.tensor([2.0, -1.0], dtype=torch.float64)) + 1)
    # lse of two terms, each a few roundings of its logarithm.
    assert (lse[:-1] - one[0]).abs().max() < 8 * 2.0 ** -24 * 2.2 and abs(lse[-1] - one[1]) < 8 * 2.0 ** -24
    assert torch.equal(loss[:-1], loss[:1].expand(n - 1))
    assert abs(loss[-1].item() - (one[1].item() + 1.0)) < 8 * 2.0 ** -24 * 1.4


@pytest.mark.parametrize("trans", [False, True])
def test_grouped_48_row_tiles(trans):
    test_grouped_every_tile(F32, trans, [90, 0, 48, 133, 90, 91, 90, 97, 96], 5003, 67)


@pytest.mark.parametrize("T,K,V", [(37, 70, 26001), (48, 130, 30000), (140, 72, 31000)])
def test_xent_48_row_tiles(T, K, V):
    test_xent_every_tile(F32, T, K, V)

"""Language-model products on the GPU: products grouped by expert and their
gradients, and the cross entropy of an output layer with its gradients,
against their definitions in float64.

Tolerances.  A bf16 result is rounded once from fp32: half a step, 2^-8 of
itself.  A sum of K products in fp32 is off by at most (K + 2) 2^-24 times the sum
of the products' magnitudes in any order (each of the additions, the product's
own rounding and the scaling by alpha contribute at most 2^-24).
"""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def padded(t, pad, shift=0):
    """The same values in rows `pad` longer, the first `shift` values into a buffer of NaN."""
    lead, (r, c) = t.shape[:-2], t.shape[-2:]
    n = r * (c + pad)
    for d in lead:
        n *= d
    buf = torch.full((n + shift + 64,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:shift + n].view(*lead, r, c + pad)[..., :c]
    v.copy_(t)
    return v


def check(out, ref, mag, n, what):
    """|out - ref| <= n 2^-24 mag, and for bf16 half a step of the value beside it."""
    out, half = out.double(), 2.0 ** -8 if out.dtype == BF16 else 0.0
    tol = n * 2.0 ** -24 * mag
    tol = tol + half * (ref.abs() + tol) + 1e-37
    bad = ~((out - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((out - ref).abs() / tol).nan_to_num(9e9).max()))


def offsets_of(sizes, first=0):
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    return ends, torch.tensor(ends, dtype=torch.int32, device="cuda")


def grouped_reference(X, W, ends, trans, alpha, beta, Y0):
    ref, mag = Y0.double().clone(), Y0.double().abs()
    for e in range(len(ends) - 1):
        a, b = ends[e], ends[e + 1]
        w = W[e].double().t() if trans else W[e].double()
        ref[a:b] = alpha * (X[a:b].double() @ w)
        mag[a:b] = abs(alpha) * (X[a:b].double().abs() @ w.abs())
        if beta:
            ref[a:b] += beta * Y0[a:b].double()
            mag[a:b] += abs(beta) * Y0[a:b].double().abs()
    return ref, mag


SIZES = {
    "one": [1], "empty": [0, 0, 0], "few": [1, 0, 2, 1], "ragged": [17, 0, 64, 1, 130, 3],
    "long": [300, 0, 513], "many": [(7 * i) % 5 for i in range(150)],
}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("N,K", [(1, 1), (64, 32), (72, 200), (131, 75), (264, 520)])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_grouped(dtype, trans, N, K, sizes):
    ends, off = offsets_of(SIZES[sizes])
    rows, E = ends[-1], len(ends) - 1
    say("grouped", dtype, trans, N, K, sizes)
    X = rand((rows, K), dtype, 1)
    W = rand((E, N, K) if trans else (E, K, N), dtype, 2)
    Y = sg.grouped_gemm(X, W, off, trans=trans)
    ref, mag = grouped_reference(X, W, ends, trans, 1.0, 0.0, torch.zeros_like(Y))
    check(Y, ref, mag, K + 2, "grouped")
    G = rand((rows, N), dtype, 3)
    D = sg.grouped_wgrad(X, G, off)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        x, g = X[a:b].double().t(), G[a:b].double()
        check(D[e], x @ g, x.abs() @ g.abs(), b - a + 2, "wgrad %d" % e)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1)])
def test_grouped_strides_scales_and_rows_outside(dtype, trans, pad, shift):
    """Padded rows, bases off alignment, alpha and beta, rows before the first and
    behind the last group left as they were, nothing written outside."""
    ends, off = offsets_of([5, 0, 40, 19], first=3)
    rows, K, N = ends[-1] + 6, 96, 80
    say("grouped strides", dtype, trans, pad, shift)
    X = padded(rand((rows, K), dtype, 1), pad, shift)
    W = padded(rand((4, N, K) if trans else (4, K, N), dtype, 2), pad, shift)
    Y0 = rand((rows, N), dtype, 3)
    Y = padded(Y0, pad, shift)
    base = Y._base.clone()
    sg.grouped_gemm(X, W, off, Y, trans=trans, alpha=-0.5, beta=2.0)
    ref, mag = grouped_reference(X, W, ends, trans, -0.5, 2.0, Y0)
    check(Y[ends[0]:ends[-1]], ref[ends[0]:ends[-1]], mag[ends[0]:ends[-1]], K + 4, "grouped")
    assert torch.equal(Y[:ends[0]], Y0[:ends[0]]) and torch.equal(Y[ends[-1]:], Y0[ends[-1]:])
    Y.copy_(Y0)
    assert torch.equal(Y._base.view(torch.int16 if dtype == BF16 else torch.int32),
                       base.view(torch.int16 if dtype == BF16 else torch.int32))
    G = padded(rand((rows, N), dtype, 4), pad, shift)
    D0 = rand((4, K, N), dtype, 5)
    D = padded(D0, pad, shift)
    sg.grouped_wgrad(X, G, off, D, alpha=1.5, beta=-1.0)
    for e in range(4):
        a, b = ends[e], ends[e + 1]
        x, g, d = X[a:b].double().t(), G[a:b].double(), D0[e].double()
        check(D[e], 1.5 * (x @ g) - d, 1.5 * (x.abs() @ g.abs()) + d.abs(), b - a + 4, "wgrad")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_values_outside_a_group_do_not_reach_it(dtype):
    """NaN and infinities in another group's rows, and in rows of no group, stay there."""
    ends, off = offsets_of([3, 2, 30], first=1)
    X, W = rand((40, 72), dtype, 1), rand((3, 72, 48), dtype, 2)
    G = rand((40, 48), dtype, 3)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[0], bad[4:6], bad[36:] = True, True, True
    X[bad], G[bad] = float("nan"), float("inf")
    Y, D = sg.grouped_gemm(X, W, off), sg.grouped_wgrad(X, G, off)
    assert not Y[~bad].isnan().any() and Y[4:6].isnan().all() and not Y[36:].any()
    assert not D[0].isnan().any() and not D[2].isnan().any() and D[1].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_without_product(dtype):
    """alpha = 0 and K = 0: Y <- beta Y, the operands unread; beta = 0 ignores old NaN."""
    _, off = offsets_of([2, 3])
    W, X = torch.full((2, 8, 8), float("nan"), dtype=dtype, device="cuda"), None
    X = torch.full((5, 8), float("nan"), dtype=dtype, device="cuda")
    Y = rand((5, 8), dtype, 1)
    Z = Y.clone()
    sg.grouped_gemm(X, W, off, Z, alpha=0.0, beta=2.0)
    assert torch.equal(Z, 2 * Y)
    sg.grouped_gemm(X[:, :0], W[:, :0], off, Z, beta=0.5)
    assert torch.equal(Z, Y)
    Z.fill_(float("nan"))
    sg.grouped_gemm(X, W, off, Z, alpha=0.0)
    assert not Z.any()
    D = torch.full((2, 8, 8), float("nan"), dtype=dtype, device="cuda")
    sg.grouped_wgrad(X, X, off, D, alpha=0.0)
    assert not D.any()
    D.fill_(float("nan"))
    sg.grouped_wgrad(X[:0], X[:0], torch.zeros(3, dtype=torch.int32, device="cuda"), D)
    assert not D.any()


def test_grouped_offsets_out_of_range_are_taken_inside():
    X, W = rand((10, 16), F32, 1), rand((4, 16, 24), F32, 2)
    off = torch.tensor([-5, 4, 2, 1 << 30, 20], dtype=torch.int32, device="cuda")
    Y = sg.grouped_gemm(X, W, off)  # groups: 0-3, none, 2-9, none
    check(Y[4:], X[4:].double() @ W[2].double(), X[4:].double().abs() @ W[2].double().abs(), 18, "y")
    D = sg.grouped_wgrad(X, Y, off)
    assert not D[1].any() and not D[3].any() and not D.isnan().any()


# ---------------------------------------------------------------- cross entropy

def xent_reference(X, W, targets, dloss=None):
    z = X.double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    counts = (targets >= 0) & (targets < W.shape[0])
    at = torch.where(counts, targets, torch.zeros_like(targets))
    loss = torch.where(counts, lse - z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    if dloss is None:
        return z, loss, lse
    d = (z - lse[:, None]).exp()
    d[torch.arange(len(at), device="cuda"), at] -= 1
    d = torch.where(counts[:, None], d * dloss.double()[:, None], torch.zeros_like(d))
    return z, loss, lse, d


def check_loss(X, W, targets, loss, lse):
    """Each logit is off by at most e = (K + 1) 2^-24 sum|x w|; lse moves by at most the
    largest e of its row, plus the roundings of the exponentials' sum: 2^-24 (V + 8) at
    most relative to the sum, so that much absolute in its logarithm, plus the last
    addition's 2^-24 |lse|.  The loss adds one more logit and one more rounding."""
    z, ref_loss, ref_lse = xent_reference(X, W, targets)
    K, V = X.shape[1], W.shape[0]
    e = (X.double().abs() @ W.double().abs().t()).amax(1) * (K + 1) * 2.0 ** -24
    # The arguments of the exponentials are rounded too: 2^-24 of their distance.
    spread = (z.amax(1) - z.amin(1)) * 2.0 ** -23
    tol = e + spread + (V + 8) * 2.0 ** -24 + 2.0 ** -23 * ref_lse.abs()
    assert ((lse.double() - ref_lse).abs() <= tol).all()
    tol = 2 * tol + 2.0 ** -23 * ref_loss.abs()
    assert ((loss.double() - ref_loss).abs() <= tol).all()


def check_gradients(X, W, targets, dloss, dX, dW, half_d=None):
    """d is off by a relative eps_d = e + 2^-23 |z - lse| + 4 2^-24 (exponent and its argument,
    e as above for the logit and again for lse), and rounded to the type: 2^-8 for bf16
    (half_d: less).  The sums over V or T then add (n + 2) 2^-24."""
    z, _, lse, d = xent_reference(X, W, targets, dloss)
    K, V, T = X.shape[1], W.shape[0], X.shape[0]
    half = 2.0 ** -8 if X.dtype == BF16 else 0.0
    e = (X.double().abs() @ W.double().abs().t()).amax(1, keepdim=True) * (K + 1) * 2.0 ** -24
    p = (z - lse[:, None]).exp() * dloss.double()[:, None].abs()
    counts = ((targets >= 0) & (targets < V))[:, None]
    off = 2 * e + ((z - lse[:, None]).abs() + (V + 16) / 2 + 2 * lse[:, None].abs()) * 2.0 ** -23
    dd = torch.where(counts, p * off, torch.zeros_like(p)) + d.abs() * ((half if half_d is None else half_d) + 2.0 ** -22)
    for out, a, b, n, what in ((dX, (d, dd), W.double(), V, "dX"), (dW, (d.t(), dd.t()), X.double(), T, "dW")):
        if out is None:
            continue
        ref = a[0] @ b
        tol = a[1] @ b.abs() + (n + 2) * 2.0 ** -24 * (a[0].abs() @ b.abs())
        tol = tol + half * (ref.abs() + tol) + 1e-37
        bad = ~((out.double() - ref).abs() <= tol)
        assert not bad.any(), "%s: %d off, worst %.3g" % (
            what, int(bad.sum()), float(((out.double() - ref).abs() / tol).nan_to_num(9e9).max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,V", [(1, 1, 1), (1, 64, 1000), (5, 40, 33), (37, 75, 1003), (130, 72, 700),
                                   (64, 136, 4100), (300, 128, 2500), (17, 256, 20011)])
def test_xent(dtype, T, K, V):
    say("xent", dtype, T, K, V)
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 2.0 / K ** 0.5)
    g = torch.Generator().manual_seed(3)
    targets = torch.randint(0, V, (T,), generator=g)
    targets[::7] = -100
    targets[3::11] = V
    targets[0] = V - 1
    targets = targets.cuda()
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    check_loss(X, W, targets, loss, lse)
    dloss = torch.rand(T, generator=g).cuda() / T
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    check_gradients(X, W, targets, dloss, dX, dW)
    one, none = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse, need_dW=False)
    assert none is None and torch.equal(one, dX)
    none, one = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse, need_dX=False)
    assert none is None and torch.equal(one, dW)

"""The language-model products with every extent zero or tiny, on the GPU."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import (BF16, F32, check, check_gradients, check_loss,  # noqa: E402
                               grouped_reference, offsets_of, rand)
from .test_q4 import check_rows  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [0, 1, 3])
def test_grouped(dtype, E):
    for rows, N, K, trans in itertools.product((0, 1, 4), (0, 1, 3), (0, 1, 3), (False, True)):
        say("edges grouped", dtype, E, rows, N, K, trans)
        ends, off = offsets_of([rows // E + (e < rows % E) for e in range(E)])
        X, W = rand((rows, K), dtype, 1), rand((E, N, K) if trans else (E, K, N), dtype, 2)
        Y = sg.grouped_gemm(X, W, off, trans=trans)
        ref, mag = grouped_reference(X, W, ends, trans, 1.0, 0.0, torch.zeros(rows, N, device="cuda"))
        check(Y, ref, mag, K + 2, "grouped")
        G = rand((rows, N), dtype, 3)
        D = sg.grouped_wgrad(X, G, off)
        assert D.shape == (E, K, N)
        for e in range(E):
            x, g = X[ends[e]:ends[e + 1]].double().t(), G[ends[e]:ends[e + 1]].double()
            check(D[e], x @ g, x.abs() @ g.abs(), rows + 2, "wgrad")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_xent(dtype):
    for T, V, K in itertools.product((0, 1, 3), (0, 1, 2, 3), (0, 1, 2, 3)):
        if V == 0 and T > 0:
            continue
        say("edges xent", dtype, T, V, K)
        X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2)
        targets = torch.arange(T, device="cuda") % max(V, 1)
        loss, lse = sg.linear_cross_entropy(X, W, targets)
        dloss = torch.ones(T, device="cuda")
        dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
        assert loss.shape == lse.shape == (T,) and dX.shape == (T, K) and dW.shape == (V, K)
        if T > 0 and K > 0:
            check_loss(X, W, targets, loss, lse)
            check_gradients(X, W, targets, dloss, dX, dW)
        elif K > 0:
            assert not dW.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_q4(dtype):
    for E, rows, N, K, block in itertools.product((None, 0, 1, 3), (0, 1, 4), (0, 1, 3), (0, 2, 34), (32, 128)):
        say("edges q4", dtype, E, rows, N, K, block)
        lead = () if E is None else (E,)
        W = rand(lead + (N, K), dtype, 1)
        Q, S, Z = sg.q4_quantize(W, block)
        assert Q.shape == lead + (N, K // 2) and S.shape == Z.shape == lead + (N, -(-K // block))
        X = rand((rows, K), dtype, 2)
        if E is None:
            Y = sg.q4_matvec(X, Q, S, Z, block=block)
            check_rows(Y, X, Q, S, Z, K, block, "q4")
            continue
        ends, off = offsets_of([rows // E + (e < rows % E) for e in range(E)])
        Y = sg.q4_matvec(X, Q, S, Z, block=block, offsets=off)
        assert Y.shape == (rows, N) and (E > 0 or not Y.any())
        for e in range(E):
            a, b = ends[e], ends[e + 1]
            check_rows(Y[a:b], X[a:b], Q[e], S[e], Z[e], K, block, "q4")

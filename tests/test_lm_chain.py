"""Two expert layers, an output layer, its loss and every gradient, on the GPU, each step
against its formula in 64 bits on what the step before it gave, so that every tolerance is
that step's own."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import (BF16, F32, check, check_gradients, check_loss,  # noqa: E402
                               grouped_reference)
from .test_lm_use import model  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_each_step(dtype):
    say("chain", dtype)
    X, A, B, O, off, ends, targets = model(dtype)
    dloss = torch.full((len(X),), 1.0 / len(X), device="cuda")

    def rows(x, w, trans, what):
        y = sg.grouped_gemm(x, w, off, trans=trans)
        ref, mag = grouped_reference(x, w, ends, trans, 1.0, 0.0, torch.zeros_like(y))
        check(y, ref, mag, x.shape[1] + 2, what)
        return y

    def weights(x, g, what):
        d = sg.grouped_wgrad(x, g, off)
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            u, v = x[a:b].double().t(), g[a:b].double()
            check(d[e], u @ v, u.abs() @ v.abs(), b - a + 2, what)

    hidden = rows(X, A, False, "first layer")
    Y = rows(hidden, B, True, "second layer")
    loss, lse = sg.linear_cross_entropy(Y, O, targets)
    check_loss(Y, O, targets, loss, lse)
    dY, dO = sg.linear_cross_entropy_backward(dloss, Y, O, targets, lse)
    # 48 rows: a bf16 derivative keeps 16 bits.
    check_gradients(Y, O, targets, dloss, dY, dO, half_d=2.0 ** -16 if dtype == BF16 else None)
    dhidden = rows(dY, B, False, "gradient of the hidden rows")
    weights(dY, hidden, "gradient of the second layer")
    rows(dhidden, A, True, "gradient of the rows")
    weights(X, dhidden, "gradient of the first layer")

"""Gradients of a mean loss, on the GPU: one dloss in every row, so that the derivatives at
the targets, all close to -dloss, round the same way in bf16."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, check_gradients, rand  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [100, 192, 384, 768])
def test_gradients_of_a_mean_loss(dtype, T):
    """Within 2^-8 of each derivative's part for more than 128 bf16 rows, 2^-16 up to that."""
    say("mean loss", dtype, T)
    K, V = 80, 3000
    X, W = rand((T, K), dtype, 1), rand((V, K), dtype, 2, 2.0 / K ** 0.5)
    targets = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    targets[::13] = -100
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    dX, dW = sg.linear_cross_entropy_backward(dloss, X, W, targets, lse)
    few = dtype == BF16 and T <= 128
    check_gradients(X, W, targets, dloss, dX, dW, half_d=2.0 ** -16 if few else None)

"""The loss of rows whose target has nearly all the probability, on the GPU.

The logits here are exact (one hidden value, a power of two), so the loss
    log(sum_v exp(z_v - z_y)) = log(1 + s),  s = sum over v != y of exp(z_v - z_y),
has no error from them.  With the target's logit the largest, the kernels' steps are off by:
the exponential of the largest value and its argument, one unit, 2^-23; adding the others to
it, whose terms may be lost whole or round up to twice (2 s) where they are below a half unit
of the sum, and otherwise half a unit each for at most 64 sums in a row that reach it; the
difference and the sum of logarithms, half a unit of values below 1 each; the logarithm, two
units of 2^-23 near 1.  In all 2 s + 16 * 2^-24 where s is far below 2^-24: nothing that
grows with the logits.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32  # noqa: E402

pytestmark = pytest.mark.gpu

ROUNDINGS = 16 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [2, 65, 700, 40000])
def test_loss_of_confident_rows(dtype, V):
    say("confident", dtype, V)
    g = torch.Generator().manual_seed(V)
    # Each row's scale is a power of two; the others lie 40 or more below its target.
    X = torch.tensor([1.0, 2.0, -1.0, 0.5] * 9, dtype=dtype)[:, None].cuda()
    best, worst = V // 3, V - 1 if V > 2 else 1
    W = (torch.rand(V, 1, generator=g) * 60 - 30).to(dtype)
    W[best], W[worst] = 231.0, -197.0
    W = W.cuda()
    targets = torch.where(X[:, 0] > 0, best, worst).cuda()
    z = X.double() @ W.double().t()
    at = z.gather(1, targets[:, None])
    s = (z - at).exp().sum(1) - 1
    assert (s < 2.0 ** -40).all() and (at > 90).all()
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    assert (loss >= 0).all()
    assert ((loss.double() - torch.log1p(s)).abs() <= 2 * s + ROUNDINGS).all(), loss


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_loss_of_a_vocabulary_of_one(dtype):
    """Its only word's loss is 0, whatever the logit."""
    X = torch.linspace(-900, 900, 301)[:, None].to(dtype).cuda()
    W = torch.tensor([[1.0]], dtype=dtype, device="cuda")
    targets = torch.zeros(301, dtype=torch.int64, device="cuda")
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    assert (loss >= 0).all() and (loss <= ROUNDINGS).all()
    assert ((lse.double() - X[:, 0].double()).abs() <= 3 * 2.0 ** -24 * X[:, 0].double().abs() + ROUNDINGS).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_loss_of_a_distant_target(dtype):
    """Two words, z apart: log(1 + exp(d)), off by two roundings of d beside the above."""
    X = torch.tensor([[1.0]], dtype=dtype, device="cuda").expand(200, 1).contiguous()
    W = torch.tensor([[500.0], [452.0]], dtype=dtype, device="cuda")
    targets = (torch.arange(200) % 2).cuda()
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    exact = torch.tensor([math.log1p(math.exp(-48)), 48.0], dtype=torch.float64, device="cuda")
    bound = torch.tensor([ROUNDINGS, ROUNDINGS + 4 * 48 * 2.0 ** -24], dtype=torch.float64, device="cuda")
    assert ((loss.double() - exact[targets]).abs() <= bound[targets]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_loss_of_infinite_logits(dtype):
    """As the definition in 64 bits has it: infinite beside an infinite logit, NaN at it."""
    inf = float("inf")
    X = torch.tensor([[1.0]], dtype=dtype, device="cuda").expand(4, 1).contiguous()
    targets = torch.tensor([0, 1, 2, -1], device="cuda")
    loss, lse = sg.linear_cross_entropy(X, torch.tensor([[1.0], [inf], [2.0]], dtype=dtype, device="cuda"), targets)
    assert (lse == inf).all() and loss[0] == inf and loss[1].isnan() and loss[2] == inf and loss[3] == 0
    loss, lse = sg.linear_cross_entropy(X, torch.tensor([[1.0], [-inf], [1.0]], dtype=dtype, device="cuda"), targets)
    assert loss[1] == inf and (loss[[0, 2]].double() - math.log(2)).abs().max() <= ROUNDINGS and loss[3] == 0
    loss, lse = sg.linear_cross_entropy(X, torch.full((3, 1), -inf, dtype=dtype, device="cuda"), targets)
    assert (lse == -inf).all() and loss[:3].isnan().all() and loss[3] == 0
    loss, lse = sg.linear_cross_entropy(X, torch.full((3, 1), float("nan"), dtype=dtype, device="cuda"), targets)
    assert loss[:3].isnan().all() and loss[3] == 0

"""Cross entropy with nothing to sum: no hidden values, no rows, a vocabulary of one."""
import math
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .conftest import ROOT  # noqa: E402
from .gpu_helpers import say  # noqa: E402
from .test_lm_abi import BACK, XENT, call  # noqa: E402
from .test_lm_products import BF16, F32  # noqa: E402


SIZES = """
import fp32_gemm_04_amd as sg
for type in (0, 1):
    for rows in (0, 1, 9, 200, 5000):
        for vocab in (0, 1, 7, 70000):
            forward, backward = (sg.sgemm_xent_workspace(type, rows, vocab, 0, b) for b in (0, 1))
            assert (forward > 0) == (rows > 0 and vocab > 0) and backward == 0, (type, rows, vocab)
"""


def test_workspace_without_hidden_values():
    """In a process of its own, since a division by zero would end it."""
    done = subprocess.run([sys.executable, "-c", SIZES], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, (done.returncode, done.stderr[-300:])


def test_backward_without_hidden_values_needs_no_workspace():
    assert call(sg.sgemm_xent_backward, BACK, dict(K=0, ws=0, ws_bytes=0)) == 0
    assert call(sg.sgemm_xent_backward, BACK, dict(ws=0, ws_bytes=0)) == -16
    assert call(sg.sgemm_xent, XENT, dict(K=0, ws=0, ws_bytes=0)) == -12


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_no_hidden_values(dtype, T):
    """Every logit is 0: the loss is log V, and the gradients have no elements."""
    say("no hidden values", dtype, T)
    V = 7
    X, W = (torch.zeros(n, 0, dtype=dtype, device="cuda") for n in (T, V))
    targets = torch.arange(T, device="cuda") % 9  # 7 and 8 do not count
    loss, lse = sg.linear_cross_entropy(X, W, targets)
    # Two units of the logarithm to base 2, and its product with log 2.
    assert (lse - math.log(7)).abs().max() <= 4 * 2.0 ** -23
    assert torch.equal(loss, torch.where(targets < V, lse, 0))
    dX, dW = sg.linear_cross_entropy_backward(torch.ones(T, device="cuda"), X, W, targets, lse)
    assert dX.shape == (T, 0) and dW.shape == (V, 0)

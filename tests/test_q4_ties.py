"""4-bit quantisation of weights that lie half way between two steps, on the GPU: the nearest
even multiple of the scale, plus the zero, whether the zero is even or odd."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .test_lm_products import BF16, F32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("zero", [None, 0, 3, 4, 15])
def test_ties(dtype, zero):
    # From -zero to 15 - zero (around 8: -7 to 7), so that the scale is 1, and all halves between.
    low = -7 if zero is None else -zero
    high = 7 if zero is None else 15 - zero
    W = torch.arange(2 * low, 2 * high + 1, device="cuda").double() / 2
    W = torch.nn.functional.pad(W, (0, 32 - len(W)))
    Q, S, Z = sg.q4_quantize(W.to(dtype)[None].contiguous(), 32, zeros=zero is not None)
    assert S.item() == 1 and (zero is None or Z.item() == zero)
    q = torch.stack([Q & 15, Q >> 4], -1).flatten()
    # torch rounds halves to even.
    assert torch.equal(q.double(), W.round() + (8 if zero is None else zero))

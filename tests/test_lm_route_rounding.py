"""What an expert layer in 8 bits rounds: with fp32 rows between the product and the weighted
sum, only the sum, on the GPU.

Tolerance.  A row's value is an exact integer sum that becomes fp32 and is multiplied by two
scales: three roundings of 2^-24.  Its product with the weight and the sum of k such terms add
(k + 1) 2^-24 of the terms' magnitudes, and the result is rounded to bf16 once: half a step,
2^-8 of itself.  Rows rounded to bf16 before the sum would add 2^-8 of every term.
"""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402
from perf import more_operators  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, check  # noqa: E402
from .test_q8 import product, quantize_reference  # noqa: E402

pytestmark = pytest.mark.gpu


def layer_reference(X, experts, weights, W, sw):
    """The layer in 64 bits from the bytes and scales of X's rows, and the sums of magnitudes."""
    Q, s = quantize_reference(X)
    ref = torch.zeros((X.shape[0], W.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e in range(len(W)):
        t, j = (experts == e).nonzero(as_tuple=True)
        v = product(Q[t], s[t], W[e], sw[e]) * weights[t, j].double()[:, None]
        ref.index_add_(0, t, v)
        mag.index_add_(0, t, v.abs())
    return ref, mag


CASES = [dict(kind="q8_experts", type=t, T=T, k=k, E=E, K=K, N=N)
         for t in ("bf16", "f32") for T, k, E, K, N in [(1, 2, 3, 64, 70), (50, 2, 5, 131, 90), (300, 2, 8, 512, 264)]]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%d" % (c["type"], c["T"]))
def test_measured_layer_rounds_its_sum_alone(case, monkeypatch):
    say("expert layer's roundings", case)
    s = more_operators.prepare(case, 3)
    monkeypatch.setattr(more_operators, "own", True)
    out = more_operators.run(s)
    assert out.dtype == s["X"].dtype
    ref, mag = layer_reference(s["X"], s["experts"], s["weights"], s["Q"], s["scales"])
    check(out, ref, mag, case["k"] + 1 + 3, "layer")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_a_choice_are_asked_for_in_either_type(dtype):
    """The product's fp32 rows rounded to bf16 are its bf16 rows: the caller chooses where."""
    s = more_operators.prepare(dict(CASES[1], type="bf16" if dtype == BF16 else "f32"), 4)
    say("rows in either type", dtype)
    offsets, _, place = sg.expert_sort(s["experts"], 5)
    Q, scales = sg.q8_quantize(s["X"], place)
    wide = sg.q8_gemm(Q, scales, s["Q"], s["scales"], offsets, dtype=F32)
    assert torch.equal(wide.to(BF16), sg.q8_gemm(Q, scales, s["Q"], s["scales"], offsets, dtype=BF16))

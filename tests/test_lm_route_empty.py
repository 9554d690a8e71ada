"""A batch without tokens, or tokens without choices, through every stage between the experts'
numbers and the layer's result."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
QUANT = dict(type=1, rows=8, K=32, X=4096, ldx=32, k=0, place=0, out_rows=8, Q=8192, ldq=32, scales=12288)


def quantize(**kw):
    return sg.sgemm_q8_quantize(*dict(QUANT, **kw).values())


@pytest.mark.parametrize("kw", [
    dict(rows=0, k=2, out_rows=0, X=0, Q=0, scales=0), dict(rows=0, k=2, out_rows=5),
    dict(rows=0, k=1, out_rows=0, K=0), dict(rows=0, k=8, out_rows=0, place=4096), dict(k=0, out_rows=0, place=4096),
])
def test_places_of_no_tokens_may_be_null(kw):
    assert quantize(**kw) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(k=2), -6), (dict(k=2, out_rows=16), -6), (dict(rows=0, k=-1, out_rows=0), -6), (dict(out_rows=0), -8),
    (dict(rows=0, out_rows=5), -8), (dict(rows=0, k=2, out_rows=-1), -8), (dict(rows=0, k=2, place=2, out_rows=0), -7),
])
def test_places_of_tokens_may_not(kw, code):
    assert quantize(**kw) == code


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k", [(0, 2), (0, 0), (5, 0)])
def test_chain(dtype, T, k):
    say("empty chain", dtype, T, k)
    E, K, N = 3, 40, 24
    X, W = torch.ones((T, K), dtype=dtype, device="cuda"), torch.ones((E, N, K), dtype=torch.int8, device="cuda")
    sw, weights = torch.ones((E, N), device="cuda"), torch.ones((T, k), device="cuda")
    offsets, order, place = sg.expert_sort(torch.zeros((T, k), dtype=torch.int64, device="cuda"), E)
    assert offsets.tolist() == [0] * 4 and order.shape == (0,) and place.shape == (T, k)
    assert sg.expert_gather(X, place, weights).shape == (0, K)
    Q, scales = sg.q8_quantize(X, place)
    assert Q.shape == (0, K) and Q.dtype == torch.int8 and scales.shape == (0,)
    rows = sg.q8_gemm(Q, scales, W, sw, offsets, dtype=dtype)
    assert rows.shape == (0, N)
    assert sg.q8_matvec(X[:0], W, sw, offsets=offsets).shape == (0, N)
    out = sg.expert_combine(rows, place, weights)
    assert out.shape == (T, N) and not out.any()
    dR, dw = sg.expert_combine_backward(out, rows, place, weights)
    assert dR.shape == (0, N) and dw.shape == (T, k)

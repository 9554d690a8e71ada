"""Operands whose sizes the calls cannot take are refused in Python, on a host without a
GPU: fake tensors have a GPU's device and any size, and no memory."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp32_gemm_04_amd as sg

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")

BIG = 2 ** 32 + 8  # as a 32-bit int: 8


def fake(*shape, dtype=torch.bfloat16, strides=None):
    if strides:
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    return torch.empty(shape, dtype=dtype, device="cuda")


def offsets(groups):
    return fake(groups + 1, dtype=torch.int32)


def targets(rows):
    return fake(rows, dtype=torch.int64)


CALLS = {
    "grouped rows": lambda: sg.grouped_gemm(fake(BIG, 4), fake(1, 4, 4), offsets(1)),
    "grouped columns": lambda: sg.grouped_gemm(fake(8, 4), fake(1, 4, BIG), offsets(1)),
    "grouped contraction": lambda: sg.grouped_gemm(fake(8, BIG), fake(1, BIG, 4), offsets(1)),
    "grouped groups": lambda: sg.grouped_gemm(fake(8, 4), fake(BIG, 4, 4), offsets(BIG)),
    "grouped leading dimension": lambda: sg.grouped_gemm(
        fake(8, 4, strides=(BIG, 1)), fake(1, 4, 4), offsets(1)),
    "grouped output": lambda: sg.grouped_gemm(
        fake(8, 4), fake(1, 4, 4), offsets(1), fake(8, 4, strides=(BIG, 1))),
    "gradient rows": lambda: sg.grouped_wgrad(fake(BIG, 4), fake(BIG, 4), offsets(1)),
    "gradient groups": lambda: sg.grouped_wgrad(fake(8, 4), fake(8, 4), offsets(BIG)),
    "gradient output": lambda: sg.grouped_wgrad(
        fake(8, 4), fake(8, 4), offsets(1), fake(1, 4, 4, strides=(1 << 40, BIG, 1))),
    "loss rows": lambda: sg.linear_cross_entropy(fake(BIG, 4), fake(9, 4), targets(BIG)),
    "loss vocabulary": lambda: sg.linear_cross_entropy(fake(8, 4), fake(BIG, 4), targets(8)),
    "loss without hidden values": lambda: sg.linear_cross_entropy(fake(8, 0), fake(BIG, 0), targets(8)),
    "4-bit rows": lambda: sg.q4_matvec(fake(BIG, 32), fake(8, 16, dtype=torch.uint8), fake(8, 1), block=32),
    "4-bit columns": lambda: sg.q4_matvec(fake(8, 32), fake(BIG, 16, dtype=torch.uint8), fake(BIG, 1), block=32),
    "quantised rows": lambda: sg.q4_quantize(fake(BIG, 2), 32),
    "quantised rows of all groups": lambda: sg.q4_quantize(fake(2 ** 20, 2 ** 12 + 1, 2), 32),
}


@pytest.mark.parametrize("call", list(CALLS))
def test_sizes_past_an_int_are_refused(call):
    with FakeTensorMode(), pytest.raises(ValueError, match="extent or stride of [0-9]{10}"):
        CALLS[call]()


@pytest.mark.parametrize("backward", [False, True])
def test_sizes_that_the_library_refuses_name_the_parameter(monkeypatch, backward):
    """Sizes that an int holds and the library does not take: its status comes back, from the
    workspace's size already."""
    monkeypatch.setattr(sg, "_current_device", lambda: 0)
    monkeypatch.setattr(sg, "_current_stream", lambda index: 0)
    with FakeTensorMode(), pytest.raises(sg.SgemmError, match="parameter 3") as e:
        X, W, t = fake(1, 0), fake(2 ** 31 - 1, 0), targets(1)
        if backward:
            row = fake(1, dtype=torch.float32)
            sg.linear_cross_entropy_backward(row, X, W, t, row)
        else:
            sg.linear_cross_entropy(X, W, t)
    assert e.value.status == -3

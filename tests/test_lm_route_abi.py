"""Host logic of the rows sorted by expert and of the 8-bit products (include/slm.h) on a host
without a GPU: argument checks before any HIP call, calls with nothing to do, workspace
sizes, and the Python functions' refusals."""
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp32_gemm_04_amd as sg

NO_GPU = not os.path.exists("/dev/kfd")
MOST = 2 ** 31 - 1025

SORT = dict(slots=64, groups=8, experts=4096, offsets=8192, order=12288, place=16384, ws=0, ws_bytes=0)
GATHER = dict(type=1, tokens=8, k=2, H=32, X=4096, ldx=32, place=8192, weights=12288, rows=16,
              R=16384, ldr=32, fill=1)
COMBINE = dict(type=1, tokens=8, k=2, H=32, rows=16, R=4096, ldr=32, place=8192, weights=12288,
               beta=0.0, out=16384, ldo=32)
BACK = dict(type=0, tokens=8, k=2, H=32, rows=16, dout=4096, lddo=32, R=8192, ldr=32, place=12288,
            weights=16384, dR=20480, lddr=32, fill=0, dweights=24576)
QUANT = dict(type=1, rows=8, K=32, X=4096, ldx=32, k=0, place=0, out_rows=8, Q=8192, ldq=32, scales=12288)
GEMM = dict(type=1, groups=1, rows=8, N=16, K=32, X=4096, ldx=32, x_scales=8192, W=12288, ldw=32,
            stride_w=512, w_scales=16384, Y=20480, ldy=16, offsets=0, fill=0)
VEC = dict(type=1, groups=1, rows=8, N=16, K=32, X=4096, ldx=32, W=12288, ldw=32, stride_w=512,
           w_scales=16384, Y=20480, ldy=16, offsets=0, fill=0)
CALLS = {"sgemm_expert_sort": SORT, "sgemm_expert_gather": GATHER, "sgemm_expert_combine": COMBINE,
         "sgemm_expert_combine_backward": BACK, "sgemm_q8_quantize": QUANT, "sgemm_q8_gemm": GEMM,
         "sgemm_q8_matvec": VEC}


def call(fn, kw):
    return getattr(sg, fn)(*dict(CALLS[fn], **kw).values())


@pytest.mark.parametrize("fn,kw,code", [
    ("sgemm_expert_sort", dict(slots=-1), -1), ("sgemm_expert_sort", dict(slots=MOST + 1), -1),
    ("sgemm_expert_sort", dict(groups=-1), -2), ("sgemm_expert_sort", dict(groups=4097), -2),
    ("sgemm_expert_sort", dict(experts=0), -3), ("sgemm_expert_sort", dict(experts=4100), -3),
    ("sgemm_expert_sort", dict(offsets=0), -4), ("sgemm_expert_sort", dict(offsets=2), -4),
    ("sgemm_expert_sort", dict(order=2), -5), ("sgemm_expert_sort", dict(place=0), -6),
    ("sgemm_expert_sort", dict(place=1), -6), ("sgemm_expert_sort", dict(slots=100000), -7),
    ("sgemm_expert_sort", dict(ws=8), -7), ("sgemm_expert_sort", dict(slots=100000, ws=4096), -8),
    ("sgemm_expert_gather", dict(type=2), -1), ("sgemm_expert_gather", dict(tokens=-1), -2),
    ("sgemm_expert_gather", dict(k=-1), -3), ("sgemm_expert_gather", dict(k=MOST // 8 + 1), -3),
    ("sgemm_expert_gather", dict(H=-1), -4), ("sgemm_expert_gather", dict(X=0), -5),
    ("sgemm_expert_gather", dict(X=4097), -5), ("sgemm_expert_gather", dict(ldx=31), -6),
    ("sgemm_expert_gather", dict(place=0), -7), ("sgemm_expert_gather", dict(place=2), -7),
    ("sgemm_expert_gather", dict(weights=2), -8), ("sgemm_expert_gather", dict(rows=-1), -9),
    ("sgemm_expert_gather", dict(R=0), -10), ("sgemm_expert_gather", dict(ldr=31), -11),
    ("sgemm_expert_gather", dict(fill=2), -12),
    ("sgemm_expert_combine", dict(type=-1), -1), ("sgemm_expert_combine", dict(tokens=MOST + 1), -2),
    ("sgemm_expert_combine", dict(k=-1), -3), ("sgemm_expert_combine", dict(H=-1), -4),
    ("sgemm_expert_combine", dict(rows=-1), -5), ("sgemm_expert_combine", dict(R=0), -6),
    ("sgemm_expert_combine", dict(ldr=31), -7), ("sgemm_expert_combine", dict(place=0), -8),
    ("sgemm_expert_combine", dict(weights=1), -9), ("sgemm_expert_combine", dict(out=0), -11),
    ("sgemm_expert_combine", dict(ldo=31), -12),
    ("sgemm_expert_combine_backward", dict(type=2), -1), ("sgemm_expert_combine_backward", dict(tokens=-1), -2),
    ("sgemm_expert_combine_backward", dict(k=-1), -3), ("sgemm_expert_combine_backward", dict(H=-1), -4),
    ("sgemm_expert_combine_backward", dict(rows=MOST + 1), -5),
    ("sgemm_expert_combine_backward", dict(dout=0), -6), ("sgemm_expert_combine_backward", dict(lddo=1), -7),
    ("sgemm_expert_combine_backward", dict(R=0), -8), ("sgemm_expert_combine_backward", dict(ldr=1), -9),
    ("sgemm_expert_combine_backward", dict(place=0), -10),
    ("sgemm_expert_combine_backward", dict(weights=2), -11),
    ("sgemm_expert_combine_backward", dict(dR=2), -12), ("sgemm_expert_combine_backward", dict(lddr=1), -13),
    ("sgemm_expert_combine_backward", dict(fill=-1), -14),
    ("sgemm_expert_combine_backward", dict(dweights=2), -15),
    ("sgemm_q8_quantize", dict(type=2), -1), ("sgemm_q8_quantize", dict(rows=-1), -2),
    ("sgemm_q8_quantize", dict(K=-1), -3), ("sgemm_q8_quantize", dict(K=131072, ldx=131072, ldq=131072), -3),
    ("sgemm_q8_quantize", dict(X=0), -4),
    ("sgemm_q8_quantize", dict(ldx=31), -5), ("sgemm_q8_quantize", dict(k=1), -6),
    ("sgemm_q8_quantize", dict(k=-1, place=4096), -6), ("sgemm_q8_quantize", dict(k=MOST, place=4096), -6),
    ("sgemm_q8_quantize", dict(k=1, place=2), -7), ("sgemm_q8_quantize", dict(out_rows=9), -8),
    ("sgemm_q8_quantize", dict(k=1, place=4096, out_rows=-1), -8),
    ("sgemm_q8_quantize", dict(Q=0), -9), ("sgemm_q8_quantize", dict(ldq=31), -10),
    ("sgemm_q8_quantize", dict(scales=0), -11), ("sgemm_q8_quantize", dict(scales=2), -11),
    ("sgemm_q8_gemm", dict(type=2), -1), ("sgemm_q8_gemm", dict(groups=2), -2),
    ("sgemm_q8_gemm", dict(groups=-1, offsets=4096), -2), ("sgemm_q8_gemm", dict(rows=-1), -3),
    ("sgemm_q8_gemm", dict(N=-1), -4), ("sgemm_q8_gemm", dict(K=131072, ldx=131072, ldw=131072), -5),
    ("sgemm_q8_gemm", dict(rows=MOST, N=MOST, ldy=2 ** 31 - 1), -4),
    ("sgemm_q8_gemm", dict(X=0), -6), ("sgemm_q8_gemm", dict(ldx=31), -7),
    ("sgemm_q8_gemm", dict(x_scales=0), -8), ("sgemm_q8_gemm", dict(W=0), -9),
    ("sgemm_q8_gemm", dict(ldw=31), -10), ("sgemm_q8_gemm", dict(stride_w=-1), -11),
    ("sgemm_q8_gemm", dict(w_scales=2), -12), ("sgemm_q8_gemm", dict(Y=20481), -13),
    ("sgemm_q8_gemm", dict(ldy=15), -14), ("sgemm_q8_gemm", dict(offsets=2), -15), ("sgemm_q8_gemm", dict(fill=2), -16),
    ("sgemm_q8_matvec", dict(type=2), -1), ("sgemm_q8_matvec", dict(groups=65536, offsets=4096), -2),
    ("sgemm_q8_matvec", dict(rows=-1), -3), ("sgemm_q8_matvec", dict(N=MOST + 1), -4),
    ("sgemm_q8_matvec", dict(K=106497, ldx=2 ** 20, ldw=2 ** 20), -5), ("sgemm_q8_matvec", dict(X=4097), -6),
    ("sgemm_q8_matvec", dict(ldx=31), -7), ("sgemm_q8_matvec", dict(W=0), -8),
    ("sgemm_q8_matvec", dict(ldw=31), -9), ("sgemm_q8_matvec", dict(stride_w=-1), -10),
    ("sgemm_q8_matvec", dict(w_scales=0), -11), ("sgemm_q8_matvec", dict(Y=0), -12),
    ("sgemm_q8_matvec", dict(ldy=15), -13), ("sgemm_q8_matvec", dict(offsets=2), -14), ("sgemm_q8_matvec", dict(fill=-1), -15),
])
def test_invalid_arguments(fn, kw, code):
    assert call(fn, kw) == code


@pytest.mark.parametrize("fn,kw", [
    ("sgemm_expert_gather", dict(tokens=0, X=0, place=0, weights=0, R=0)),
    ("sgemm_expert_gather", dict(H=0, X=0, place=0, R=0)),
    ("sgemm_expert_gather", dict(rows=0, X=0, place=0, R=0)),
    ("sgemm_expert_combine", dict(tokens=0, R=0, place=0, out=0)),
    ("sgemm_expert_combine", dict(H=0, R=0, place=0, out=0)),
    ("sgemm_expert_combine_backward", dict(k=0, dout=0, R=0, place=0)),
    ("sgemm_expert_combine_backward", dict(dR=0, dweights=0, dout=0, R=0, place=0)),
    ("sgemm_expert_combine_backward", dict(H=0, dweights=0, dout=0, R=0, place=0)),
    ("sgemm_q8_quantize", dict(rows=0, out_rows=0, X=0, Q=0, scales=0)),
    ("sgemm_q8_quantize", dict(place=4096, k=0, X=0, Q=0, scales=0)),
    ("sgemm_q8_gemm", dict(rows=0, X=0, x_scales=0, W=0, w_scales=0, Y=0)),
    ("sgemm_q8_gemm", dict(N=0, X=0, x_scales=0, W=0, w_scales=0, Y=0)),
    ("sgemm_q8_gemm", dict(groups=0, offsets=4096, X=0, W=0, Y=0)),
    ("sgemm_q8_matvec", dict(rows=0, X=0, W=0, w_scales=0, Y=0)),
    ("sgemm_q8_matvec", dict(N=0, X=0, W=0, w_scales=0, Y=0)),
])
def test_nothing_to_do_needs_no_pointers(fn, kw):
    assert call(fn, kw) == 0


@pytest.mark.skipif(not NO_GPU, reason="a GPU device node is present")
@pytest.mark.parametrize("fn", list(CALLS))
def test_valid_arguments_reach_the_device(fn):
    assert call(fn, {}) > 0  # the checks pass; HIP reports no device


def test_sort_workspace():
    size = sg.sgemm_expert_sort_workspace
    assert size(-1, 1) == -1 and size(MOST + 1, 1) == -1 and size(1, -1) == -2 and size(1, 4097) == -2
    assert size(0, 0) == 0 and size(16384, 64) == 0  # one launch needs none
    assert size(16385, 64) == 20 * 65 * 4  # seventeen chunks of 1024, rounded up to four
    assert size(65537, 2000) == 36 * 2001 * 4  # many experts: 33 chunks of 2048
    assert size(MOST, 4096) == 256 * 4097 * 4  # never more than 256 segments


def fake(*shape, dtype=torch.bfloat16, strides=None):
    if strides:
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    return torch.empty(shape, dtype=dtype, device="cuda")


I8, I32, I64, F32, BIG = torch.int8, torch.int32, torch.int64, torch.float32, 2 ** 32 + 8
REFUSED = {
    "experts' type": (TypeError, lambda: sg.expert_sort(fake(4, 2, dtype=I32), 3)),
    "experts' shape": (TypeError, lambda: sg.expert_sort(fake(4, dtype=I64), 3)),
    "experts not packed": (ValueError, lambda: sg.expert_sort(fake(4, 2, dtype=I64, strides=(3, 1)), 3)),
    "experts past an int": (ValueError, lambda: sg.expert_sort(fake(BIG, 1, dtype=I64), 3)),
    "groups past an int": (ValueError, lambda: sg.expert_sort(fake(4, 1, dtype=I64), BIG)),
    "place's type": (ValueError, lambda: sg.expert_gather(fake(4, 8), fake(4, 2, dtype=I64))),
    "place's rows": (ValueError, lambda: sg.expert_gather(fake(4, 8), fake(5, 2, dtype=I32))),
    "place's shape": (ValueError, lambda: sg.expert_gather(fake(4, 8), fake(4, dtype=I32))),
    "place not packed": (ValueError, lambda: sg.expert_gather(fake(4, 8), fake(4, 2, dtype=I32, strides=(4, 1)))),
    "weights' type": (ValueError, lambda: sg.expert_gather(fake(4, 8), fake(4, 2, dtype=I32), fake(4, 2))),
    "weights' shape": (ValueError, lambda: sg.expert_combine(fake(8, 8), fake(4, 2, dtype=I32), fake(4, 3, dtype=F32))),
    "rows' type": (TypeError, lambda: sg.expert_combine(fake(8, 8, dtype=torch.half), fake(4, 2, dtype=I32))),
    "column stride": (ValueError, lambda: sg.expert_gather(fake(4, 8, strides=(1, 4)), fake(4, 2, dtype=I32))),
    "rows overlap": (ValueError, lambda: sg.expert_gather(fake(4, 8, strides=(7, 1)), fake(4, 2, dtype=I32))),
    "out's columns": (ValueError, lambda: sg.expert_gather(fake(4, 8), fake(4, 2, dtype=I32), out=fake(8, 9))),
    "out's rows": (ValueError, lambda: sg.expert_combine(fake(8, 8), fake(4, 2, dtype=I32), out=fake(5, 8))),
    "dout's type": (TypeError, lambda: sg.expert_combine_backward(fake(4, 8, dtype=F32), fake(8, 8), fake(4, 2, dtype=I32))),
    "dR's rows": (ValueError, lambda: sg.expert_combine_backward(
        fake(4, 8), fake(8, 8), fake(4, 2, dtype=I32), dR=fake(9, 8))),
    "quantised type": (TypeError, lambda: sg.q8_quantize(fake(4, 8, dtype=I8))),
    "quantised groups to rows": (TypeError, lambda: sg.q8_quantize(fake(2, 4, 8), fake(4, 2, dtype=I32))),
    "quantised groups apart": (ValueError, lambda: sg.q8_quantize(fake(2, 4, 8, strides=(64, 8, 1)))),
    "quantised rows past an int": (ValueError, lambda: sg.q8_quantize(fake(2 ** 20, 2 ** 12, 1))),
    "quantised place": (ValueError, lambda: sg.q8_quantize(fake(4, 8), fake(3, 2, dtype=I32))),
    "bytes' type": (TypeError, lambda: sg.q8_gemm(fake(4, 8), fake(4, dtype=F32), fake(6, 8, dtype=I8), fake(6, dtype=F32))),
    "row scales": (ValueError, lambda: sg.q8_gemm(fake(4, 8, dtype=I8), fake(5, dtype=F32), fake(6, 8, dtype=I8), fake(6, dtype=F32))),
    "column scales": (ValueError, lambda: sg.q8_gemm(fake(4, 8, dtype=I8), fake(4, dtype=F32), fake(6, 8, dtype=I8), fake(7, dtype=F32))),
    "contractions": (ValueError, lambda: sg.q8_gemm(fake(4, 8, dtype=I8), fake(4, dtype=F32), fake(6, 9, dtype=I8), fake(6, dtype=F32))),
    "groups without offsets": (ValueError, lambda: sg.q8_matvec(fake(4, 8), fake(2, 6, 8, dtype=I8), fake(2, 6, dtype=F32))),
    "one set with offsets": (ValueError, lambda: sg.q8_matvec(
        fake(4, 8), fake(6, 8, dtype=I8), fake(6, dtype=F32), offsets=fake(2, dtype=I32))),
    "offsets": (ValueError, lambda: sg.q8_matvec(
        fake(4, 8), fake(2, 6, 8, dtype=I8), fake(2, 6, dtype=F32), offsets=fake(2, dtype=I32))),
    "result's type": (TypeError, lambda: sg.q8_gemm(
        fake(4, 8, dtype=I8), fake(4, dtype=F32), fake(6, 8, dtype=I8), fake(6, dtype=F32), dtype=torch.half)),
    "result's shape": (ValueError, lambda: sg.q8_matvec(
        fake(4, 8), fake(6, 8, dtype=I8), fake(6, dtype=F32), Y=fake(4, 7))),
}


@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
@pytest.mark.parametrize("what", list(REFUSED))
def test_python_refuses(what):
    error, refused = REFUSED[what]
    with FakeTensorMode(), pytest.raises(error):
        refused()


def test_operands_on_the_host_are_refused():
    X, place = torch.zeros(4, 8), torch.zeros(4, 2, dtype=I32)
    for fn in (lambda: sg.expert_sort(torch.zeros(4, 2, dtype=I64), 3), lambda: sg.expert_gather(X, place),
               lambda: sg.expert_combine(X, place), lambda: sg.expert_combine_backward(X, X, place),
               lambda: sg.q8_quantize(X), lambda: sg.q8_matvec(X, X.to(I8), X[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            fn()

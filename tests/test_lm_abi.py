"""Host logic of the language-model products (include/slm.h) on a host without a
GPU: argument checks come before any HIP call, calls with nothing to do make
none, and the Python functions refuse operands that do not fit together."""
import os

import pytest
import torch

import fp32_gemm_04_amd as sg

NO_GPU = not os.path.exists("/dev/kfd")

GROUPED = dict(type=1, trans=0, groups=2, rows=8, N=32, K=16, alpha=1.0, X=4096, ldx=16, W=8192,
               ldw=32, stride_w=512, beta=0.0, Y=12288, ldy=32, offsets=16384)
WGRAD = dict(type=1, groups=2, rows=8, M=16, N=32, alpha=1.0, X=4096, ldx=16, G=8192, ldg=32,
             beta=0.0, D=12288, ldd=32, stride_d=512, offsets=16384)
XENT = dict(type=0, rows=8, vocab=100, K=16, X=4096, ldx=16, W=8192, ldw=16, targets=12288,
            loss=16384, lse=16640, ws=20480, ws_bytes=1 << 20)
BACK = dict(type=0, rows=8, vocab=100, K=16, X=4096, ldx=16, W=8192, ldw=16, targets=12288,
            lse=16640, dloss=16384, dX=20480, lddx=16, dW=24576, lddw=16, ws=32768,
            ws_bytes=1 << 20)
Q4 = dict(type=1, groups=1, rows=3, N=32, K=64, block=32, X=4096, ldx=64, Q=8192, S=12288, Z=16384,
          Y=20480, ldy=32, offsets=0)
QUANT = dict(type=1, N=32, K=64, block=32, W=4096, ldw=64, Q=8192, S=12288, Z=16384)


def call(fn, good, kw):
    args = dict(good)
    args.update(kw)
    return fn(*args.values())


@pytest.mark.parametrize("fn,good,kw,code", [
    ("sgemm_grouped", GROUPED, dict(type=2), -1), ("sgemm_grouped", GROUPED, dict(trans=2), -2),
    ("sgemm_grouped", GROUPED, dict(groups=-1), -3), ("sgemm_grouped", GROUPED, dict(rows=-1), -4),
    ("sgemm_grouped", GROUPED, dict(N=-1), -5), ("sgemm_grouped", GROUPED, dict(K=-1), -6),
    ("sgemm_grouped", GROUPED, dict(X=0), -8), ("sgemm_grouped", GROUPED, dict(X=4097), -8),
    ("sgemm_grouped", GROUPED, dict(ldx=15), -9), ("sgemm_grouped", GROUPED, dict(W=0), -10),
    ("sgemm_grouped", GROUPED, dict(ldw=31), -11),
    ("sgemm_grouped", GROUPED, dict(trans=1, ldw=15), -11),
    ("sgemm_grouped", GROUPED, dict(stride_w=-1), -12), ("sgemm_grouped", GROUPED, dict(Y=0), -14),
    ("sgemm_grouped", GROUPED, dict(ldy=31), -15), ("sgemm_grouped", GROUPED, dict(offsets=0), -16),
    ("sgemm_grouped", GROUPED, dict(offsets=16386), -16),
    ("sgemm_grouped", GROUPED, dict(rows=2 ** 31 - 1025, N=2 ** 31 - 1025, ldw=2 ** 31 - 1,
                                    ldy=2 ** 31 - 1), -5),
    ("sgemm_grouped", GROUPED, dict(rows=2 ** 31 - 1024), -4),
    ("sgemm_grouped", GROUPED, dict(K=2 ** 31 - 1024), -6),
    ("sgemm_grouped_wgrad", WGRAD, dict(M=2 ** 31 - 1024), -4),
    ("sgemm_xent", XENT, dict(vocab=2 ** 31 - 1024), -3),
    ("sgemm_grouped_wgrad", WGRAD, dict(type=-1), -1),
    ("sgemm_grouped_wgrad", WGRAD, dict(groups=-1), -2),
    ("sgemm_grouped_wgrad", WGRAD, dict(rows=-1), -3),
    ("sgemm_grouped_wgrad", WGRAD, dict(M=-1), -4), ("sgemm_grouped_wgrad", WGRAD, dict(N=-1), -5),
    ("sgemm_grouped_wgrad", WGRAD, dict(X=0), -7), ("sgemm_grouped_wgrad", WGRAD, dict(ldx=1), -8),
    ("sgemm_grouped_wgrad", WGRAD, dict(G=0), -9), ("sgemm_grouped_wgrad", WGRAD, dict(ldg=1), -10),
    ("sgemm_grouped_wgrad", WGRAD, dict(D=0), -12), ("sgemm_grouped_wgrad", WGRAD, dict(ldd=1), -13),
    ("sgemm_grouped_wgrad", WGRAD, dict(stride_d=-1), -14),
    ("sgemm_grouped_wgrad", WGRAD, dict(offsets=0), -15),
    ("sgemm_xent", XENT, dict(type=7), -1), ("sgemm_xent", XENT, dict(rows=-1), -2),
    ("sgemm_xent", XENT, dict(vocab=0), -3), ("sgemm_xent", XENT, dict(K=-1), -4),
    ("sgemm_xent", XENT, dict(X=0), -5), ("sgemm_xent", XENT, dict(ldx=15), -6),
    ("sgemm_xent", XENT, dict(W=8194), -7), ("sgemm_xent", XENT, dict(ldw=15), -8),
    ("sgemm_xent", XENT, dict(targets=12292), -9), ("sgemm_xent", XENT, dict(loss=0), -10),
    ("sgemm_xent", XENT, dict(lse=0), -11), ("sgemm_xent", XENT, dict(ws=20484), -12),
    ("sgemm_xent", XENT, dict(ws_bytes=100), -13),
    ("sgemm_xent_backward", BACK, dict(targets=0), -9),
    ("sgemm_xent_backward", BACK, dict(lse=0), -10),
    ("sgemm_xent_backward", BACK, dict(dloss=2), -11),
    ("sgemm_xent_backward", BACK, dict(dX=20482), -12),
    ("sgemm_xent_backward", BACK, dict(lddx=15), -13),
    ("sgemm_xent_backward", BACK, dict(dW=24577), -14),
    ("sgemm_xent_backward", BACK, dict(ws_bytes=16), -17),
    ("sgemm_xent_backward", BACK, dict(lddw=15), -15), ("sgemm_xent_backward", BACK, dict(ws=0), -16),
    ("sgemm_q4_matvec", Q4, dict(type=3), -1), ("sgemm_q4_matvec", Q4, dict(groups=2), -2),
    ("sgemm_q4_matvec", Q4, dict(groups=65536, offsets=16384), -2),
    ("sgemm_q4_matvec", Q4, dict(rows=-1), -3), ("sgemm_q4_matvec", Q4, dict(N=-1), -4),
    ("sgemm_q4_matvec", Q4, dict(K=2 ** 27 + 2, ldx=2 ** 28), -5),
    ("sgemm_q4_matvec", Q4, dict(K=63), -5), ("sgemm_q4_matvec", Q4, dict(block=16), -6),
    ("sgemm_q4_matvec", Q4, dict(X=0), -7), ("sgemm_q4_matvec", Q4, dict(ldx=63), -8),
    ("sgemm_q4_matvec", Q4, dict(Q=0), -9), ("sgemm_q4_matvec", Q4, dict(S=1), -10),
    ("sgemm_q4_matvec", Q4, dict(Y=0), -12), ("sgemm_q4_matvec", Q4, dict(ldy=31), -13),
    ("sgemm_q4_matvec", Q4, dict(offsets=2), -14),
    ("sgemm_q4_quantize", QUANT, dict(type=3), -1), ("sgemm_q4_quantize", QUANT, dict(N=-1), -2),
    ("sgemm_q4_quantize", QUANT, dict(K=1), -3), ("sgemm_q4_quantize", QUANT, dict(block=0), -4),
    ("sgemm_q4_quantize", QUANT, dict(W=0), -5), ("sgemm_q4_quantize", QUANT, dict(ldw=63), -6),
    ("sgemm_q4_quantize", QUANT, dict(Q=0), -7), ("sgemm_q4_quantize", QUANT, dict(S=0), -8),
])
def test_invalid_arguments(fn, good, kw, code):
    assert call(getattr(sg, fn), good, kw) == code


@pytest.mark.parametrize("fn,good,kw", [
    ("sgemm_grouped", GROUPED, dict(groups=0, X=0, W=0, Y=0, offsets=0)),
    ("sgemm_grouped", GROUPED, dict(rows=0, X=0, W=0, Y=0, offsets=0)),
    ("sgemm_grouped", GROUPED, dict(N=0, X=0, W=0, Y=0, offsets=0)),
    ("sgemm_grouped_wgrad", WGRAD, dict(groups=0, X=0, G=0, D=0, offsets=0)),
    ("sgemm_grouped_wgrad", WGRAD, dict(M=0, X=0, G=0, D=0, offsets=0)),
    ("sgemm_xent", XENT, dict(rows=0, X=0, W=0, targets=0, loss=0, lse=0, ws=0, ws_bytes=0)),
    ("sgemm_xent_backward", BACK, dict(dX=0, dW=0)),
    ("sgemm_xent_backward", BACK, dict(K=0, dX=0, dW=0)),
    ("sgemm_xent_backward", BACK, dict(rows=0, dW=0, X=0, targets=0, lse=0, dloss=0, ws=0)),
    ("sgemm_q4_matvec", Q4, dict(rows=0, X=0, Q=0, S=0, Y=0)),
    ("sgemm_q4_matvec", Q4, dict(N=0, X=0, Q=0, S=0, Y=0)),
    ("sgemm_q4_quantize", QUANT, dict(N=0, W=0, Q=0, S=0)),
    ("sgemm_q4_quantize", QUANT, dict(K=0, W=0, Q=0, S=0)),
])
def test_nothing_to_do_needs_no_pointers(fn, good, kw):
    assert call(getattr(sg, fn), good, kw) == 0


@pytest.mark.skipif(not NO_GPU, reason="a GPU device node is present")
@pytest.mark.parametrize("fn,good", [
    ("sgemm_grouped", GROUPED), ("sgemm_grouped_wgrad", WGRAD), ("sgemm_xent", XENT),
    ("sgemm_xent_backward", BACK), ("sgemm_q4_matvec", Q4), ("sgemm_q4_quantize", QUANT),
])
def test_valid_arguments_reach_the_device(fn, good):
    assert call(getattr(sg, fn), good, {}) > 0  # the checks pass; HIP reports no device


def test_workspace_sizes():
    assert sg.sgemm_xent_workspace(2, 1, 1, 1, 0) == -1
    assert sg.sgemm_xent_workspace(0, -1, 1, 1, 0) == -2
    assert sg.sgemm_xent_workspace(0, 1, -1, 1, 0) == -3
    assert sg.sgemm_xent_workspace(0, 1, 1, -1, 0) == -4
    assert sg.sgemm_xent_workspace(0, 1, 1, 1, 2) == -5
    assert sg.sgemm_xent_workspace(0, 0, 10, 10, 1) == 0
    # Never the logits: a long batch over a large vocabulary keeps one piece at a time.
    T, V, H = 65536, 131072, 4096
    assert 0 < sg.sgemm_xent_workspace(1, T, V, H, 1) < T * V * 2 / 8
    assert 0 < sg.sgemm_xent_workspace(1, T, V, H, 0) < T * V * 2 / 8


def test_python_refuses_what_does_not_fit():
    X = torch.zeros(4, 8)
    off = torch.zeros(3, dtype=torch.int32)
    for fn, args in [(sg.grouped_gemm, (X, torch.zeros(2, 8, 5), off)),
                     (sg.grouped_wgrad, (X, X, off)),
                     (sg.linear_cross_entropy, (X, torch.zeros(9, 8), torch.zeros(4).long())),
                     (sg.q4_matvec, (X, torch.zeros(5, 4, dtype=torch.uint8), torch.zeros(5, 1))),
                     (sg.q4_quantize, (X,))]:
        with pytest.raises(ValueError, match="GPU"):
            fn(*args)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sg.grouped_gemm(X.double(), X, off)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sg.linear_cross_entropy(X.half(), X, off)


def test_errors_name_the_call():
    assert "sgemm_xent failed with status -5: invalid parameter 5" in str(sg.SgemmError(-5, "sgemm_xent"))
    assert "invalid M" in str(sg.SgemmError(-1))


@pytest.mark.parametrize("ldd,stride_d,code", [
    (32, 0, -14), (32, 511, -14), (64, 31, -14), (65, 34, -14),  # groups that share elements
    (32, 512, 0), (64, 32, 0), (65, 33, 0), (32, 1 << 62, 0)])
def test_wgrad_outputs_must_not_overlap(ldd, stride_d, code):
    args = dict(WGRAD, ldd=ldd, stride_d=stride_d)
    if code == 0:
        args["offsets"] = 0  # the next check, so that no call reaches a device
        code = -15
    assert sg.sgemm_grouped_wgrad(*args.values()) == code
    assert sg.sgemm_grouped_wgrad(*dict(args, groups=1, offsets=0).values()) == -15

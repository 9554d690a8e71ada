"""Python binding of libsgemm, the MI355X single-precision GEMM.

Argument marshalling only: every step of the product runs in the HIP
kernels of ``libsgemm.so`` (built from ``csrc/`` by ``_build.py``).  If the
library is missing, importing this package raises; there is no fallback.

The functions have the names and arguments of the C ABI in
``include/sgemm.h``; ``gemm`` is a convenience that takes torch tensors and
passes their data pointers, leading dimensions and the current stream.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libsgemm.so")

SGEMM_VARIANT_AUTO = 0
SGEMM_VARIANT_MFMA = 1
SGEMM_VARIANT_VALU = 2
SGEMM_VARIANT_SKINNY = 3
SGEMM_VARIANT_MFMA_TILE = 16
SGEMM_VARIANT_LADDER = 32
SGEMM_VARIANT_STREAMK_TILE = 48
SGEMM_LADDER_RUNGS = 8
LADDER_RUNG_NAMES = ("naive", "coalesced", "lds", "tile1d", "tile2d", "regcache", "vec4", "dbuf")
SGEMM_ERR_BAD_VARIANT = -100
SGEMM_ERR_VARIANT_SHAPE = -101
SGEMM_ERR_WORKSPACE = -102
SGEMM_ERR_NO_SLOT = -103
SGEMM_ERR_CAPTURING = -104

SGEMM_TYPE_F32 = 0
SGEMM_TYPE_BF16 = 1

SCONV_VARIANT_AUTO = 0
SCONV_VARIANT_STEM = 1
SCONV_VARIANT_GENERAL = 2
SCONV_VARIANT_TILE = 3
SCONV_VARIANT_DIRECT = 4
SCONV_VARIANT_TAP = 5

EXPORTS = ("sgemm_f32", "sgemm_f32_variant", "sgemm_plan", "sgemm_tune", "sgemm_tune_reset",
           "sgemm_num_mfma_tiles", "sgemm_status_string",
           # include/sconv.h
           "sconv2d_f32", "sconv2d_f32_variant", "sgemm_im2col_f32", "sconv2d_plan",
           "sconv2d_num_stem_kernels",
           # include/slm.h
           "sgemm_grouped", "sgemm_grouped_wgrad", "sgemm_xent", "sgemm_xent_backward",
           "sgemm_xent_workspace", "sgemm_q4_matvec", "sgemm_q4_quantize")

if not os.path.exists(LIBRARY):
    raise ImportError("libsgemm.so is not built; run __graft_entry__.build() "
                      "(or python fp32_gemm_04_amd/_build.py)")

# torch must be loaded first.  Its wheel carries its own HIP runtime
# (libamdhip64, soname libamdhip64.so.7, found through torch's RPATH as
# "libamdhip64.so"); libsgemm asks for "libamdhip64.so.7", which then
# resolves to that same already-loaded runtime.  Loaded the other way round,
# the process would hold two HIP runtimes, and torch's streams and memory
# would be foreign to the one libsgemm calls.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIBRARY)

_gemm_args = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
              ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
              ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
_lib.sgemm_f32.restype = ctypes.c_int
_lib.sgemm_f32.argtypes = _gemm_args
_lib.sgemm_f32_variant.restype = ctypes.c_int
_lib.sgemm_f32_variant.argtypes = [ctypes.c_int] + _gemm_args
_lib.sgemm_plan.restype = ctypes.c_int
_lib.sgemm_plan.argtypes = [ctypes.c_int] * 7 + [ctypes.c_float, ctypes.c_int,
                                                 ctypes.c_char_p, ctypes.c_int]
_lib.sgemm_tune.restype = ctypes.c_int
_lib.sgemm_tune.argtypes = _gemm_args + [ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_float)]
_lib.sgemm_tune_reset.restype = None
_lib.sgemm_tune_reset.argtypes = []
_lib.sgemm_num_mfma_tiles.restype = ctypes.c_int
_lib.sgemm_num_mfma_tiles.argtypes = []
_lib.sgemm_status_string.restype = ctypes.c_char_p
_lib.sgemm_status_string.argtypes = [ctypes.c_int]
_conv_args = ([ctypes.c_int] * 11 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_void_p])
_lib.sconv2d_f32.restype = ctypes.c_int
_lib.sconv2d_f32.argtypes = _conv_args
_lib.sconv2d_f32_variant.restype = ctypes.c_int
_lib.sconv2d_f32_variant.argtypes = [ctypes.c_int] + _conv_args
_lib.sgemm_im2col_f32.restype = ctypes.c_int
_lib.sgemm_im2col_f32.argtypes = ([ctypes.c_int] * 10 + [ctypes.c_void_p, ctypes.c_void_p,
                                                         ctypes.c_int, ctypes.c_void_p])
_lib.sconv2d_plan.restype = ctypes.c_int
_lib.sconv2d_plan.argtypes = [ctypes.c_int] * 13 + [ctypes.c_char_p, ctypes.c_int]
_lib.sconv2d_num_stem_kernels.restype = ctypes.c_int
_lib.sconv2d_num_stem_kernels.argtypes = []
_i, _i64, _f, _p = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
for _name, _args in {
        "sgemm_grouped": [_i] * 6 + [_f, _p, _i, _p, _i, _i64, _f, _p, _i, _p, _p],
        "sgemm_grouped_wgrad": [_i] * 5 + [_f, _p, _i, _p, _i, _f, _p, _i, _i64, _p, _p],
        "sgemm_xent": [_i] * 4 + [_p, _i, _p, _i, _p, _p, _p, _p, _i64, _p],
        "sgemm_xent_backward": [_i] * 4 + [_p, _i, _p, _i] + [_p] * 4 + [_i, _p, _i, _p, _i64, _p],
        "sgemm_q4_matvec": [_i] * 6 + [_p, _i, _p, _p, _p, _p, _i, _p, _p],
        "sgemm_q4_quantize": [_i] * 4 + [_p, _i, _p, _p, _p, _p],
}.items():
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = _args
_lib.sgemm_xent_workspace.restype = ctypes.c_int64
_lib.sgemm_xent_workspace.argtypes = [ctypes.c_int] * 5


class SgemmError(RuntimeError):
    """A non-zero status; ``call`` names the entry point whose header says what
    -p means where it is not sgemm_f32's list."""

    def __init__(self, status: int, call: str = ""):
        if call and -100 < status < 0:
            text = "%s failed with status %d: invalid parameter %d" % (call, status, -status)
        else:
            text = "%s failed with status %d: %s" % (call or "sgemm", status,
                                                      sgemm_status_string(status))
        super().__init__(text)
        self.status = status


def sgemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """C ABI ``sgemm_f32``; pointers and stream are integers.  Returns the status."""
    return _lib.sgemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_f32_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """C ABI ``sgemm_f32_variant``.  Returns the status."""
    return _lib.sgemm_f32_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_plan(variant, M, N, K, lda, ldb, ldc, alpha, num_cus):
    """C ABI ``sgemm_plan``.  Returns (status, text)."""
    buf = ctypes.create_string_buffer(256)
    rc = _lib.sgemm_plan(variant, M, N, K, lda, ldb, ldc, alpha, num_cus, buf, len(buf))
    return rc, buf.value.decode()


def sgemm_tune(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0, reps=5):
    """C ABI ``sgemm_tune``.  Returns (status, chosen variant, microseconds per launch)."""
    chosen = ctypes.c_int(0)
    us = ctypes.c_float(0.0)
    rc = _lib.sgemm_tune(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, reps,
                         ctypes.byref(chosen), ctypes.byref(us))
    return rc, chosen.value, us.value


def sgemm_tune_reset() -> None:
    """C ABI ``sgemm_tune_reset``."""
    _lib.sgemm_tune_reset()


def sgemm_num_mfma_tiles() -> int:
    """C ABI ``sgemm_num_mfma_tiles``."""
    return _lib.sgemm_num_mfma_tiles()


def sgemm_status_string(status: int) -> str:
    return _lib.sgemm_status_string(status).decode()


def tune(A, B, C, alpha: float = 1.0, beta: float = 0.0, reps: int = 5, stream=None):
    """Tune the kernel choice for this problem (``sgemm_tune``) and compute
    C <- alpha*A@B + beta*C in place with the winner.  Returns (variant,
    microseconds per launch); raises SgemmError on a non-zero status."""
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape), tuple(C.shape)))
    s = stream if stream is not None else torch.cuda.current_stream(C.device)
    rc, chosen, us = sgemm_tune(M, N, K, alpha, A.data_ptr(), _ld(A, "A"), B.data_ptr(),
                                _ld(B, "B"), beta, C.data_ptr(), _ld(C, "C"), s.cuda_stream, reps)
    if rc != 0:
        raise SgemmError(rc)
    return chosen, us


def _ld(t, name):
    if t.dim() != 2 or t.dtype.__repr__() != "torch.float32":
        raise TypeError("%s must be a 2-D float32 tensor" % name)
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    if t.shape[0] > 1 and t.numel():
        return t.stride(0)
    return max(1, t.shape[1])


def gemm(A, B, C, alpha: float = 1.0, beta: float = 0.0, variant: int = SGEMM_VARIANT_AUTO,
         stream=None):
    """C <- alpha*A@B + beta*C in place, for float32 CUDA/HIP tensors.

    Rows may be padded (stride(0) >= columns).  Queues on ``stream`` (a
    torch stream) or the current stream; raises SgemmError on a non-zero
    status.
    """
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape), tuple(C.shape)))
    s = stream if stream is not None else torch.cuda.current_stream(C.device)
    rc = _lib.sgemm_f32_variant(variant, M, N, K, alpha, A.data_ptr(), _ld(A, "A"),
                                B.data_ptr(), _ld(B, "B"), beta, C.data_ptr(), _ld(C, "C"),
                                s.cuda_stream)
    if rc != 0:
        raise SgemmError(rc)
    return C


# ------------------------------------------------------------ convolution

def sconv2d_f32(batch, channels, height, width, out_channels, kernel_h, kernel_w, stride_h,
                stride_w, pad_h, pad_w, alpha, X, Wt, ldw, beta, Y, ldy, stream=0) -> int:
    """C ABI ``sconv2d_f32``; pointers and stream are integers.  Returns the status."""
    return _lib.sconv2d_f32(batch, channels, height, width, out_channels, kernel_h, kernel_w,
                            stride_h, stride_w, pad_h, pad_w, alpha, X, Wt, ldw, beta, Y, ldy,
                            stream)


def sconv2d_f32_variant(variant, batch, channels, height, width, out_channels, kernel_h,
                        kernel_w, stride_h, stride_w, pad_h, pad_w, alpha, X, Wt, ldw, beta, Y,
                        ldy, stream=0) -> int:
    """C ABI ``sconv2d_f32_variant``.  Returns the status."""
    return _lib.sconv2d_f32_variant(variant, batch, channels, height, width, out_channels,
                                    kernel_h, kernel_w, stride_h, stride_w, pad_h, pad_w, alpha,
                                    X, Wt, ldw, beta, Y, ldy, stream)


def sgemm_im2col_f32(batch, channels, height, width, kernel_h, kernel_w, stride_h, stride_w,
                     pad_h, pad_w, X, B, ldb, stream=0) -> int:
    """C ABI ``sgemm_im2col_f32``.  Returns the status."""
    return _lib.sgemm_im2col_f32(batch, channels, height, width, kernel_h, kernel_w, stride_h,
                                 stride_w, pad_h, pad_w, X, B, ldb, stream)


def sconv2d_plan(variant, batch, channels, height, width, out_channels, kernel_h, kernel_w,
                 stride_h, stride_w, pad_h, pad_w, num_cus):
    """C ABI ``sconv2d_plan``.  Returns (status, text)."""
    buf = ctypes.create_string_buffer(256)
    rc = _lib.sconv2d_plan(variant, batch, channels, height, width, out_channels, kernel_h,
                           kernel_w, stride_h, stride_w, pad_h, pad_w, num_cus, buf, len(buf))
    return rc, buf.value.decode()


def sconv2d_num_stem_kernels() -> int:
    """C ABI ``sconv2d_num_stem_kernels``."""
    return _lib.sconv2d_num_stem_kernels()


def _pair(v):
    return (v, v) if isinstance(v, int) else tuple(v)


def conv2d(X, Wt, kernel, stride=1, pad=0, Y=None, alpha: float = 1.0, beta: float = 0.0,
           variant: int = SCONV_VARIANT_AUTO, stream=None):
    """Y <- alpha * conv(X, filters) + beta * Y for float32 device tensors:
    X packed (batch, C, H, W); Wt the filters as an out_channels x (C*R*S)
    matrix (or (out_channels, C, R, S), packed); Y an out_channels x
    (batch*OH*OW) matrix (allocated, zero, when None).  Returns Y; raises
    SgemmError on a non-zero status."""
    import torch
    R, S = _pair(kernel)
    sh, sw = _pair(stride)
    ph, pw = _pair(pad)
    batch, C, H, W = X.shape
    if not X.is_contiguous():
        raise ValueError("X must be packed NCHW")
    M = Wt.shape[0]
    W2 = Wt.reshape(M, -1) if Wt.dim() == 4 else Wt
    OH = (H + 2 * ph - R) // sh + 1
    OW = (W + 2 * pw - S) // sw + 1
    if Y is None:
        Y = torch.zeros((M, batch * OH * OW), dtype=torch.float32, device=X.device)
    s = stream if stream is not None else torch.cuda.current_stream(X.device)
    rc = _lib.sconv2d_f32_variant(variant, batch, C, H, W, M, R, S, sh, sw, ph, pw, alpha,
                                  X.data_ptr(), W2.data_ptr(), _ld(W2, "Wt"), beta, Y.data_ptr(),
                                  _ld(Y, "Y"), s.cuda_stream)
    if rc != 0:
        raise SgemmError(rc)
    return Y


def im2col(X, kernel, stride=1, pad=0, B=None, stream=None):
    """The (C*R*S) x (batch*OH*OW) im2col matrix of a packed NCHW float32
    device tensor (into B, allocated when None).  Returns B."""
    import torch
    R, S = _pair(kernel)
    sh, sw = _pair(stride)
    ph, pw = _pair(pad)
    batch, C, H, W = X.shape
    if not X.is_contiguous():
        raise ValueError("X must be packed NCHW")
    OH = (H + 2 * ph - R) // sh + 1
    OW = (W + 2 * pw - S) // sw + 1
    if B is None:
        B = torch.empty((C * R * S, batch * OH * OW), dtype=torch.float32, device=X.device)
    s = stream if stream is not None else torch.cuda.current_stream(X.device)
    rc = _lib.sgemm_im2col_f32(batch, C, H, W, R, S, sh, sw, ph, pw, X.data_ptr(), B.data_ptr(),
                               _ld(B, "B"), s.cuda_stream)
    if rc != 0:
        raise SgemmError(rc)
    return B


# ---------------------------------------------- language-model products

def sgemm_grouped(type, trans, groups, rows, N, K, alpha, X, ldx, W, ldw, stride_w, beta, Y, ldy,
                  offsets, stream=0) -> int:
    """C ABI ``sgemm_grouped``; pointers and stream are integers.  Returns the status."""
    return _lib.sgemm_grouped(type, trans, groups, rows, N, K, alpha, X, ldx, W, ldw, stride_w,
                              beta, Y, ldy, offsets, stream)


def sgemm_grouped_wgrad(type, groups, rows, M, N, alpha, X, ldx, G, ldg, beta, D, ldd, stride_d,
                        offsets, stream=0) -> int:
    """C ABI ``sgemm_grouped_wgrad``.  Returns the status."""
    return _lib.sgemm_grouped_wgrad(type, groups, rows, M, N, alpha, X, ldx, G, ldg, beta, D, ldd,
                                    stride_d, offsets, stream)


def sgemm_xent(type, rows, vocab, K, X, ldx, W, ldw, targets, loss, lse, ws, ws_bytes,
               stream=0) -> int:
    """C ABI ``sgemm_xent``.  Returns the status."""
    return _lib.sgemm_xent(type, rows, vocab, K, X, ldx, W, ldw, targets, loss, lse, ws, ws_bytes,
                           stream)


def sgemm_xent_backward(type, rows, vocab, K, X, ldx, W, ldw, targets, lse, dloss, dX, lddx, dW,
                        lddw, ws, ws_bytes, stream=0) -> int:
    """C ABI ``sgemm_xent_backward``.  Returns the status."""
    return _lib.sgemm_xent_backward(type, rows, vocab, K, X, ldx, W, ldw, targets, lse, dloss, dX,
                                    lddx, dW, lddw, ws, ws_bytes, stream)


def sgemm_xent_workspace(type, rows, vocab, K, backward) -> int:
    """C ABI ``sgemm_xent_workspace``: bytes, or a negative status."""
    return _lib.sgemm_xent_workspace(type, rows, vocab, K, backward)


def sgemm_q4_matvec(type, groups, rows, N, K, block, X, ldx, Q, S, Z, Y, ldy, offsets,
                    stream=0) -> int:
    """C ABI ``sgemm_q4_matvec``.  Returns the status."""
    return _lib.sgemm_q4_matvec(type, groups, rows, N, K, block, X, ldx, Q, S, Z, Y, ldy, offsets,
                                stream)


def sgemm_q4_quantize(type, N, K, block, W, ldw, Q, S, Z, stream=0) -> int:
    """C ABI ``sgemm_q4_quantize``.  Returns the status."""
    return _lib.sgemm_q4_quantize(type, N, K, block, W, ldw, Q, S, Z, stream)


_TYPES = {torch.float32: SGEMM_TYPE_F32, torch.bfloat16: SGEMM_TYPE_BF16}


_MOST_INT = 2 ** 31 - 1  # ctypes passes larger numbers on without their high bits


def _extent(n, name):
    if n > _MOST_INT:
        raise ValueError("%s has an extent or stride of %d: the calls take int" % (name, n))
    return n


def _operand(t, name, dtype, device, dim=2, rows=None, cols=None):
    """Checks a tensor of rows with unit column stride; returns its leading dimension."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != dim:
        raise TypeError("%s must be a %d-D %s tensor, not %d-D %s"
                        % (name, dim, dtype, len(shape), t.dtype))
    if not t.is_cuda or t.device != device:
        raise ValueError("%s is on %s: every operand must be on one GPU" % (name, t.device))
    r, c = shape[-2], shape[-1]
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError("%s is %s: %s x %s is wanted" % (name, tuple(shape), rows, cols))
    if r > _MOST_INT or c > _MOST_INT or shape[0] > _MOST_INT:
        _extent(max(shape), name)
    if t.is_contiguous():
        return c if c > 1 else 1
    if t.numel() == 0:
        return max(1, c)
    if c > 1 and t.stride(-1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    if r > 1:
        if t.stride(-2) < c:
            raise ValueError("%s has overlapping rows" % name)
        return _extent(t.stride(-2), name)
    return max(1, c)


def _groups_of(t):
    """Elements from one group's matrix to the next."""
    return t.stride(0) if t.shape[0] > 1 else 0


def _vector(t, name, dtype, device, n):
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a packed %s vector of %d on %s" % (name, dtype, n, device))
    return t.data_ptr()


def _type_of(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, not %s" % (name, t.dtype))
    return code


_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(call, device, stream, operands, body):
    """body(stream handle) with ``device`` current and, where a stream is given,
    with it current too, so that what body allocates belongs to that stream;
    the operands' memory is then kept from reuse until that stream is past the call."""
    if stream is None and device.index == _current_device():
        rc = body(_current_stream(device.index))  # the usual case, without context managers
    else:
        if stream is not None and stream.device != device:
            raise ValueError("the stream is on %s, the operands on %s" % (stream.device, device))
        with torch.cuda.device(device):
            if stream is None:
                rc = body(_current_stream(device.index))
            else:
                with torch.cuda.stream(stream):
                    rc = body(stream.cuda_stream)
                for t in operands:
                    if t is not None:
                        t.record_stream(stream)
    if rc != 0:
        raise SgemmError(rc, call)


def grouped_gemm(X, W, offsets, Y=None, trans: bool = False, alpha: float = 1.0,
                 beta: float = 0.0, stream=None):
    """Y[r] <- alpha * X[r] @ W[e] + beta * Y[r] for the rows r of each group e,
    offsets[e] <= r < offsets[e + 1] (``sgemm_grouped``).

    X: (rows, K); W: (groups, K, N), or (groups, N, K) with ``trans``; offsets:
    groups + 1 int32 on the device, increasing; Y: (rows, N), allocated as
    zeros when None (a pass over Y of its own).  float32 or bfloat16, rows may be
    padded.  Rows outside every group keep what Y holds.  Autograd does not see the
    product: its gradients are ``grouped_gemm(dY, W, offsets, trans=not trans)`` and
    ``grouped_wgrad``.  Returns Y.
    """
    t = _type_of(X, "X")
    dev = X.device
    ldx = _operand(X, "X", X.dtype, dev)
    rows, K = X.shape
    if W.dim() != 3:
        raise TypeError("W must be 3-D")
    groups, N = W.shape[0], W.shape[1 if trans else 2]
    ldw = _operand(W, "W", X.dtype, dev, 3, *((N, K) if trans else (K, N)))
    off = _vector(offsets, "offsets", torch.int32, dev, groups + 1)
    ldy = _operand(Y, "Y", X.dtype, dev, 2, rows, N) if Y is not None else max(1, N)

    def body(s):
        nonlocal Y
        if Y is None:
            Y = X.new_zeros(rows, N)
        return _lib.sgemm_grouped(t, int(trans), groups, rows, N, K, alpha, X.data_ptr(), ldx,
                                  W.data_ptr(), ldw, _groups_of(W), beta, Y.data_ptr(), ldy, off, s)
    _run("sgemm_grouped", dev, stream, (X, W, offsets, Y), body)
    return Y


def grouped_wgrad(X, G, offsets, D=None, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """D[e] <- alpha * X_e^T @ G_e + beta * D[e] over each group's rows
    (``sgemm_grouped_wgrad``): the gradient of grouped weights.

    X: (rows, M); G: (rows, N); offsets as in ``grouped_gemm``; D: (groups, M,
    N), allocated as zeros when None.  For weights stored (K, N): X is the
    product's input and G its output's gradient; for weights stored (N, K),
    exchange the two.  Returns D.
    """
    t = _type_of(X, "X")
    dev = X.device
    ldx = _operand(X, "X", X.dtype, dev)
    rows, M = X.shape
    ldg = _operand(G, "G", X.dtype, dev, 2, rows)
    N = G.shape[1]
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be a vector of groups + 1 row numbers")
    groups = _extent(offsets.shape[0] - 1, "offsets")
    off = _vector(offsets, "offsets", torch.int32, dev, groups + 1)
    if D is not None and D.shape[0] != groups:
        raise ValueError("D has %d groups, offsets %d" % (D.shape[0], groups))
    ldd = _operand(D, "D", X.dtype, dev, 3, M, N) if D is not None else max(1, N)

    def body(s):
        nonlocal D
        if D is None:
            D = (X.new_empty if beta == 0.0 else X.new_zeros)(groups, M, N)
        return _lib.sgemm_grouped_wgrad(t, groups, rows, M, N, alpha, X.data_ptr(), ldx,
                                        G.data_ptr(), ldg, beta, D.data_ptr(), ldd, _groups_of(D),
                                        off, s)
    _run("sgemm_grouped_wgrad", dev, stream, (X, G, offsets, D), body)
    return D


def _xent_operands(X, W, targets):
    t = _type_of(X, "X")
    dev = X.device
    ldx = _operand(X, "X", X.dtype, dev)
    rows, K = X.shape
    ldw = _operand(W, "W", X.dtype, dev, 2, None, K)
    vocab = W.shape[0]
    if vocab == 0 and rows > 0:
        raise ValueError("W holds no vocabulary")
    return t, dev, ldx, ldw, rows, K, vocab, _vector(targets, "targets", torch.int64, dev, rows)


def linear_cross_entropy(X, W, targets, stream=None):
    """(loss, lse) of each row of X: the softmax cross entropy of the logits
    X @ W.T at ``targets``, and the logits' log-sum-exp (``sgemm_xent``).  The
    logits are not kept.

    X: (rows, K); W: (vocab, K), float32 or bfloat16; targets: int64, one per
    row; a target outside [0, vocab) marks a row that does not count (loss 0).
    loss and lse are float32.  Autograd does not see them: the gradients are
    ``linear_cross_entropy_backward``'s.
    """
    t, dev, ldx, ldw, rows, K, vocab, tg = _xent_operands(X, W, targets)
    loss = lse = None

    def body(s):
        nonlocal loss, lse
        loss, lse = (X.new_empty(rows, dtype=torch.float32) for _ in range(2))
        n = _lib.sgemm_xent_workspace(t, rows, vocab, K, 0)
        if n < 0:
            return n
        ws = X.new_empty(n, dtype=torch.uint8)
        return _lib.sgemm_xent(t, rows, vocab, K, X.data_ptr(), ldx, W.data_ptr(), ldw, tg,
                               loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), n, s)
    _run("sgemm_xent", dev, stream, (X, W, targets), body)
    return loss, lse


def linear_cross_entropy_backward(dloss, X, W, targets, lse, dX=None, dW=None, need_dX: bool = True,
                                  need_dW: bool = True, stream=None):
    """(dX, dW): gradients of sum(dloss * loss) of ``linear_cross_entropy`` by X
    and W (``sgemm_xent_backward``).  dloss: float32, one per row; lse as the
    forward pass gave it; dX and dW are allocated when None; one that is not
    needed is not computed and comes back as None.
    """
    t, dev, ldx, ldw, rows, K, vocab, tg = _xent_operands(X, W, targets)
    pl = _vector(lse, "lse", torch.float32, dev, rows)
    pd = _vector(dloss, "dloss", torch.float32, dev, rows)
    lddx = _operand(dX, "dX", X.dtype, dev, 2, rows, K) if dX is not None else max(1, K)
    lddw = _operand(dW, "dW", X.dtype, dev, 2, vocab, K) if dW is not None else max(1, K)
    dX, dW = dX if need_dX else None, dW if need_dW else None

    def body(s):
        nonlocal dX, dW
        if need_dX and dX is None:
            dX = X.new_empty(rows, K)
        if need_dW and dW is None:
            dW = X.new_empty(vocab, K)
        n = _lib.sgemm_xent_workspace(t, rows, vocab, K, 1)
        if n < 0:
            return n
        ws = X.new_empty(n, dtype=torch.uint8)
        return _lib.sgemm_xent_backward(t, rows, vocab, K, X.data_ptr(), ldx, W.data_ptr(), ldw, tg,
                                        pl, pd, dX.data_ptr() if need_dX else 0, lddx,
                                        dW.data_ptr() if need_dW else 0, lddw, ws.data_ptr(), n, s)
    _run("sgemm_xent_backward", dev, stream, (dloss, X, W, targets, lse, dX, dW), body)
    return dX, dW


Q4_BLOCKS = (32, 64, 128)


def _packed(t, name, dtype, device, shape):
    if t.dtype is not dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a packed %s tensor of %s on %s" % (name, dtype, shape, device))
    return t.data_ptr()


def q4_quantize(W, block: int = 128, zeros: bool = True, stream=None):
    """(Q, scales, zeros): W in 4 bits with a scale, and with ``zeros`` a zero, for
    each ``block`` (32, 64 or 128) of weights along K (``sgemm_q4_quantize``).

    W: (N, K) or (groups, N, K), packed groups, float32 or bfloat16, values below 2^127
    in magnitude, K even.  Q: uint8 of (..., N,
    K/2), two weights a byte, the even one in the low half; scales: W's type,
    (..., N, ceil(K/block)); zeros: uint8 likewise, or None.
    """
    t = _type_of(W, "W")
    dev, lead, (N, K) = W.device, tuple(W.shape[:-2]), W.shape[-2:]
    ldw = _operand(W, "W", W.dtype, dev, W.dim())
    if W.dim() not in (2, 3):
        raise TypeError("W must be 2-D or 3-D")
    if block not in Q4_BLOCKS:
        raise ValueError("block must be one of %s" % (Q4_BLOCKS,))
    if K % 2:
        raise ValueError("K must be even")
    if W.dim() == 3 and W.shape[0] > 1 and W.numel() and W.stride(0) != N * ldw:
        raise ValueError("W's groups must follow one another")
    blocks = -(-K // block)
    rows = _extent(N * (lead[0] if lead else 1), "W as one matrix")
    Q = S = Z = None

    def body(s):
        nonlocal Q, S, Z
        Q = W.new_empty(lead + (N, K // 2), dtype=torch.uint8)
        S = W.new_empty(lead + (N, blocks))
        Z = W.new_empty(lead + (N, blocks), dtype=torch.uint8) if zeros else None
        return _lib.sgemm_q4_quantize(t, rows, K, block, W.data_ptr(), ldw, Q.data_ptr(),
                                      S.data_ptr(), Z.data_ptr() if zeros else 0, s)
    _run("sgemm_q4_quantize", dev, stream, (W,), body)
    return Q, S, Z


def q4_matvec(X, Q, scales, zeros=None, block: int = 128, Y=None, offsets=None, stream=None):
    """Y[r] <- X[r] @ w.T with weights held in 4 bits, w[n, k] = (q[n, k] - zero) *
    scale of the row's block (``sgemm_q4_matvec``), for a few rows.

    X: (rows, K), float32 or bfloat16; Q, scales, zeros as ``q4_quantize`` gives
    them (zeros None: 8); Y: (rows, N), allocated when None.  With ``offsets``
    (groups + 1 int32), Q, scales and zeros hold one set of weights per group, and
    row r uses its group's; rows outside every group keep what Y holds.
    """
    t = _type_of(X, "X")
    dev = X.device
    ldx = _operand(X, "X", X.dtype, dev)
    rows, K = X.shape
    if block not in Q4_BLOCKS:
        raise ValueError("block must be one of %s" % (Q4_BLOCKS,))
    if K % 2:
        raise ValueError("K must be even")
    *lead, N, bytes_ = Q.shape if Q.dim() > 1 else (0, 0, 0, 0)
    if len(lead) != (0 if offsets is None else 1):
        raise ValueError("Q must be (N, K/2), or (groups, N, K/2) with offsets")
    groups = lead[0] if lead else 1
    if bytes_ != K // 2:
        raise ValueError("Q holds %d weights a row, X %d values" % (2 * bytes_, K))
    per_block = (*lead, N, -(-K // block))
    pq = _packed(Q, "Q", torch.uint8, dev, Q.shape)
    _extent(N if N > groups else groups, "Q")
    ps = _packed(scales, "scales", X.dtype, dev, per_block)
    pz = _packed(zeros, "zeros", torch.uint8, dev, per_block) if zeros is not None else 0
    off = _vector(offsets, "offsets", torch.int32, dev, groups + 1) if offsets is not None else 0
    ldy = _operand(Y, "Y", X.dtype, dev, 2, rows, N) if Y is not None else max(1, N)

    def body(s):
        nonlocal Y
        if Y is None:
            Y = (X.new_empty if offsets is None else X.new_zeros)(rows, N)
        return _lib.sgemm_q4_matvec(t, groups, rows, N, K, block, X.data_ptr(), ldx, pq, ps, pz,
                                    Y.data_ptr(), ldy, off, s)
    _run("sgemm_q4_matvec", dev, stream, (X, Q, scales, zeros, Y, offsets), body)
    return Y

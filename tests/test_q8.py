"""Products in 8-bit integers on the GPU.  Quantisation is compared value by value with exact
rational rounding in float64 (its quotient of two fp32 values tells every tie of a half
integer apart: 2^-53 against a distance of at least 2^-32), products with exact integer sums.

Tolerance.  The exact sum is below 2^31 and becomes fp32, is multiplied by two scales and
rounded to the type: three roundings of 2^-24 of the value, and 2^-8 of it for bf16.
"""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import check, offsets_of, padded, rand  # noqa: E402
from .test_lm_route import routed  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PART = torch.tensor(1 / 127, dtype=F32).item()  # products of two 24-bit numbers are exact in 64 bits


def quantize_reference(X):
    X = X.double()
    finite = torch.isfinite(X).all(1)
    m = X.abs().amax(1) if X.shape[1] else X.new_zeros(X.shape[0])
    scales = (m * PART).float()
    q = torch.round(X / scales.double()[:, None])
    q = torch.where((scales > 0)[:, None] & finite[:, None], q, 0.0).nan_to_num(0.0).clamp(-127, 127)
    return q.to(torch.int8), torch.where(finite, scales, float("nan"))


def assert_quantized(X, Q, scales):
    q, s = quantize_reference(X)
    assert torch.equal(scales.nan_to_num(-1.0), s.nan_to_num(-1.0))
    assert torch.equal(Q, q), int((Q != q).sum())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 15), (5, 16), (9, 17), (64, 1024), (7, 1025), (6, 2048),
                                    (5, 2050), (3, 4096), (2, 10007), (300, 64), (0, 8), (4, 0)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_quantize(dtype, rows, K, pad, shift):
    say("quantize", dtype, rows, K, pad, shift)
    X = padded(rand((rows, K), dtype, 1), pad, shift) if rows * K else rand((rows, K), dtype, 1)
    Q, scales = sg.q8_quantize(X)
    assert Q.shape == X.shape and (Q.stride(0) % 16 == 0 or rows < 2 or K == 0)
    assert_quantized(X, Q, scales)


def test_quantize_rounds_the_exact_quotient():
    """Values at and next to half steps, for scales of every leading digits: what a product
    with the reciprocal, or a rounded quotient, gets wrong."""
    say("quantize ties")
    m = torch.cat([torch.arange(1, 4096, dtype=torch.float64) / 2048, torch.tensor([127.0, 254.0, 1 / 3])])
    m = m.float()
    s = (m.double() * PART).float().double()
    steps = torch.arange(0, 127, dtype=torch.float64) + 0.5
    mid = (s[:, None] * steps).float()
    near = [mid, torch.nextafter(mid, torch.zeros(())), torch.nextafter(mid, torch.tensor(9e9))]
    X = torch.cat(near + [m[:, None]], 1)
    X = torch.cat([X, -X]).clamp(-m.repeat(2)[:, None], m.repeat(2)[:, None]).cuda()
    assert_quantized(X, *sg.q8_quantize(X))
    exact = torch.cat([torch.tensor([127.0]), torch.arange(-127, 127) + 0.5]).view(1, -1).cuda()  # scale 1
    Q = sg.q8_quantize(exact)[0][0].tolist()
    assert Q[0] == 127 and Q[1:5] == [-126, -126, -124, -124] and all(q % 2 == 0 for q in Q[1:])


def test_quantize_of_tiny_huge_and_missing_values():
    say("quantize extremes")
    tiny, inf, nan = 2.0 ** -149, float("inf"), float("nan")
    rows = [[0.0] * 4, [tiny, -tiny, 0.0, tiny], [190 * tiny, -64 * tiny, 63 * tiny, 0.0],
            [127 * tiny, 3 * tiny, -50 * tiny, tiny], [1e-38, -3e-39, 1e-42, 0.0], [1e-30, 3e-31, -1e-33, 0.0],
            [3.4e38, -1.7e38, 1e30, 1.0], [1.0, inf, 0.0, 2.0], [-inf, 1.0, 1.0, 1.0], [nan, 1.0, 2.0, 3.0],
            [1.0, -0.0, 0.0, 0.0039], [2.0 ** -60, 2.0 ** -61, 1e-20, -2.0 ** -67]]
    X = torch.tensor(rows, dtype=torch.float64).float().cuda()
    assert X[1, 0] > 0
    Q, scales = sg.q8_quantize(X)
    assert_quantized(X, Q, scales)
    assert torch.isnan(scales[7:10]).all() and (Q[7:10] == 0).all()
    Y = sg.q8_gemm(Q, scales, torch.ones(2, 4, dtype=torch.int8, device="cuda"), torch.ones(2, device="cuda"), dtype=F32)
    assert torch.isnan(Y[7:10]).all() and torch.isfinite(Y[:7]).all()
    V = sg.q8_matvec(X, torch.ones(2, 4, dtype=torch.int8, device="cuda"), torch.ones(2, device="cuda"))
    assert torch.equal(V.nan_to_num(-7.0), Y.nan_to_num(-7.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,K", [(1, 1, 1), (40, 2, 100), (9, 8, 2048), (5, 3, 5003), (4, 2, 17001)])
def test_quantize_to_sorted_rows(dtype, T, k, K):
    say("quantize to rows", dtype, T, k, K)
    _, order, place, _ = routed(T, k, 6, T + K, 0.2)
    X = rand((T, K), dtype, 2)
    Q0, s0 = sg.q8_quantize(X)
    Q, s = sg.q8_quantize(X, place)
    held = place.flatten()[order] >= 0
    assert torch.equal(Q, torch.where(held[:, None], Q0[order // k], torch.zeros_like(Q)))
    assert torch.equal(s, torch.where(held, s0[order // k], torch.zeros_like(s)))


def test_quantize_of_all_experts_weights():
    say("quantize groups")
    W = rand((3, 20, 72), BF16, 1)
    Q, s = sg.q8_quantize(W)
    assert Q.shape == W.shape and s.shape == (3, 20)
    for e in range(3):
        assert_quantized(W[e], Q[e], s[e])


def bytes_of(shape, seed, low=-128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def positive(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda") + 0.25


def product(X, sx, W, sw):
    """The exact sums (float64 holds them) times the scales."""
    return (X.double() @ W.double().t()) * sx.double()[:, None] * sw.double()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 1), (1, 70, 130), (16, 64, 128), (17, 65, 127), (40, 200, 500),
                                      (100, 131, 1000), (130, 260, 96), (257, 300, 144), (1030, 1100, 272),
                                      (5, 33, 0), (0, 8, 8), (8, 0, 8), (3, 50, 4099), (30, 7, 0)])
@pytest.mark.parametrize("pad", [0, 4, 3])
def test_gemm(dtype, rows, N, K, pad):
    say("q8 gemm", dtype, rows, N, K, pad)
    X = bytes_of((rows, K + pad), 1)[:, :K]
    W = bytes_of((N, K + pad), 2)[:, :K]
    sx, sw = positive((rows,), 3), positive((N,), 4)
    ref = product(X, sx, W, sw)
    check(sg.q8_gemm(X, sx, W, sw, dtype=dtype), ref, ref.abs(), 3, "product")
    if rows and N:
        Y = padded(torch.zeros((rows, N), dtype=dtype, device="cuda"), pad, 1)
        base = Y._base.clone()
        sg.q8_gemm(X, sx, W, sw, Y=Y)
        check(Y, ref, ref.abs(), 3, "padded")
        Y.zero_()
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(Y._base.view(bits), base.view(bits))


def test_longest_sums_do_not_overflow():
    say("q8 longest")
    K = 131071
    X = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    W = torch.stack([X[0], -(X[0] + 1)])  # -128, and 127
    one = torch.ones(2, device="cuda")
    Y = sg.q8_gemm(X, one, W, one, dtype=F32)
    assert Y.tolist() == [[float(K * 16384), float(-K * 128 * 127)]] * 2
    with pytest.raises(sg.SgemmError, match="parameter 5"):
        sg.q8_gemm(bytes_of((1, K + 1), 1), one[:1], bytes_of((1, K + 1), 2), one[:1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[1], [0, 0], [1, 0, 2, 1], [17, 0, 64, 1, 130, 3], [300, 0, 513],
                                   [(7 * i) % 5 for i in range(150)]])
@pytest.mark.parametrize("N,K,pad", [(1, 1, 3), (72, 200, 0), (131, 75, 0), (264, 520, 8)])
def test_grouped(dtype, sizes, N, K, pad):
    say("q8 grouped", dtype, sizes[:4], N, K, pad)
    ends, off = offsets_of(sizes, first=2)
    rows, E = ends[-1] + 3, len(sizes)
    X = bytes_of((rows, K + pad), 1)[:, :K]
    W = bytes_of((E, N, K + pad), 2)[..., :K]
    sx, sw = positive((rows,), 3), positive((E, N), 4)
    Y0 = rand((rows, N), dtype, 5)
    Y = Y0.clone()
    sg.q8_gemm(X, sx, W, sw, off, Y)
    ref = Y0.double()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        ref[a:b] = product(X[a:b], sx[a:b], W[e], sw[e])
    check(Y, ref, ref.abs(), 3, "grouped")
    assert torch.equal(Y[:2], Y0[:2]) and torch.equal(Y[-3:], Y0[-3:])
    # The same rows from values, quantised inside the product.
    V0 = rand((rows, K), dtype, 6)
    V = sg.q8_matvec(V0, W, sw, Y0.clone(), off)
    Q, s = sg.q8_quantize(V0)
    assert torch.equal(V, sg.q8_gemm(Q, s, W, sw, off, Y0.clone()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 15, 16, 17, 40])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (50, 129), (200, 1000), (33, 1111), (4100, 512), (40, 8192)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 1)])
def test_matvec(dtype, rows, N, K, pad, shift):
    say("q8 matvec", dtype, rows, N, K, pad, shift)
    X = padded(rand((rows, K), dtype, 1), pad, shift)
    W = bytes_of((N, K + pad), 2)[:, :K]
    sw = positive((N,), 3)
    Y = sg.q8_matvec(X, W, sw)
    Q, s = sg.q8_quantize(X)
    ref = product(Q, s, W, sw)
    check(Y, ref, ref.abs(), 3, "matvec")
    assert torch.equal(Y, sg.q8_gemm(Q, s, W, sw, dtype=dtype))
    into = padded(torch.zeros((rows, N), dtype=dtype, device="cuda"), pad, shift)
    base = into._base.clone()
    assert sg.q8_matvec(X, W, sw, into) is into and torch.equal(into, Y)
    into.zero_()
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(into._base.view(bits), base.view(bits))


def one_launch(X, W, sw, offsets=None):
    """sgemm_q8_matvec whatever the number of values (q8_matvec quantises many beforehand)."""
    groups, N, (rows, K) = W.shape[0] if W.dim() == 3 else 1, W.shape[-2], X.shape
    Y = torch.full((rows, N), float("nan"), dtype=X.dtype, device="cuda")
    status = sg.sgemm_q8_matvec(
        int(X.dtype == BF16), groups, rows, N, K, X.data_ptr(), X.stride(0), W.data_ptr(), W.stride(-2),
        W.stride(0) if W.dim() == 3 else 0, sw.data_ptr(), Y.data_ptr(), N,
        offsets.data_ptr() if offsets is not None else 0, 1, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    return Y


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K", [(1, 106496), (3, 50000), (16, 7000), (9, 9000), (2, 106496), (16, 4096),
                                    (40, 1200), (1, 40000)])
@pytest.mark.parametrize("pad", [0, 2])
def test_matvec_of_long_rows_takes_passes(dtype, rows, K, pad):
    say("q8 matvec long", dtype, rows, K, pad)
    X, W, sw = rand((rows, K), dtype, 1), bytes_of((37, K + pad), 2)[:, :K], positive((37,), 3)
    Q, s = sg.q8_quantize(X)
    ref = sg.q8_gemm(Q, s, W, sw, dtype=dtype)
    assert torch.equal(one_launch(X, W, sw), ref) and torch.equal(sg.q8_matvec(X, W, sw), ref)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[0, 0, 0], [3, 0, 40], [16, 17, 1, 0], [0] * 70 + [2, 0, 1] + [0] * 60 + [5],
                                   [0] * 63 + [1, 1] + [0] * 200, [1] + [0] * 9])
def test_matvec_of_groups_fills_rows_outside(dtype, sizes):
    """In one launch and in two; rows outside every group become zero where the result is allocated."""
    say("q8 matvec groups", dtype, sizes)
    ends, off = offsets_of(sizes, first=3)
    for K in (200, 3000):
        X, W, sw = rand((ends[-1] + 4, K), dtype, 1), bytes_of((len(sizes), 70, K), 2), positive((len(sizes), 70), 3)
        Q, s = sg.q8_quantize(X)
        ref = torch.zeros((X.shape[0], 70), dtype=torch.float64, device="cuda")
        for e in range(len(sizes)):
            a, b = ends[e], ends[e + 1]
            ref[a:b] = product(Q[a:b], s[a:b], W[e], sw[e])
        for Y in (one_launch(X, W, sw, off), sg.q8_matvec(X, W, sw, offsets=off),
                  sg.q8_gemm(Q, s, W, sw, off, dtype=dtype)):
            check(Y, ref, ref.abs(), 3, "groups")


@pytest.mark.parametrize("rows", [0, 3, 40])
@pytest.mark.parametrize("groups", [0, 5])
def test_products_without_a_contraction(rows, groups):
    say("q8 K 0", rows, groups)
    X = torch.empty((rows, 0), dtype=BF16, device="cuda")
    W = torch.empty(((groups,) if groups else ()) + (70, 0), dtype=torch.int8, device="cuda")
    sw, off = positive(W.shape[:-1], 1), offsets_of([0, rows] + [0] * 3)[1] if groups else None
    Q, s = sg.q8_quantize(X)
    assert Q.shape == (rows, 0) and not s.any()
    for Y in (sg.q8_matvec(X, W, sw, offsets=off), sg.q8_gemm(Q, s, W, sw, off)):
        assert Y.shape == (rows, 70) and not Y.any()


def test_matvec_of_more_groups_than_a_grid_has():
    groups, K, N = 65540, 20, 3
    say("q8 matvec groups", groups)
    sizes = [0] * groups
    sizes[0], sizes[40], sizes[-1] = 2, 1, 3
    ends, off = offsets_of(sizes)
    X, W, sw = rand((6, K), BF16, 1), bytes_of((groups, N, K), 2), positive((groups, N), 3)
    Q, s = sg.q8_quantize(X)
    group = torch.tensor([0, 0, 40] + [groups - 1] * 3, device="cuda")
    ref = torch.stack([product(Q[r:r + 1], s[r:r + 1], W[g], sw[g])[0] for r, g in enumerate(group.tolist())])
    Y = sg.q8_matvec(X, W, sw, offsets=off)
    check(Y, ref, ref.abs(), 3, "groups")
    assert torch.equal(Y, sg.q8_gemm(Q, s, W, sw, off))


def test_no_groups_at_all():
    say("q8 no groups")
    X, off = rand((5, 32), BF16, 1), torch.tensor([2], dtype=torch.int32, device="cuda")
    W, sw = torch.empty((0, 9, 32), dtype=torch.int8, device="cuda"), torch.empty((0, 9), device="cuda")
    Q, s = sg.q8_quantize(X)
    for Y in (sg.q8_matvec(X, W, sw, offsets=off), sg.q8_gemm(Q, s, W, sw, off)):
        assert Y.shape == (5, 9) and (Y == 0).all()


def test_matvec_over_many_tiles():
    """More tiles of columns than one set of their scales covers (32 a workgroup)."""
    N, K = 16 * 512 * 70 + 5, 40
    say("q8 matvec wide", N)
    X, W, sw = rand((2, K), F32, 1), bytes_of((N, K), 2), positive((N,), 3)
    Q, s = sg.q8_quantize(X)
    ref = product(Q, s, W, sw)
    check(sg.q8_matvec(X, W, sw), ref, ref.abs(), 3, "wide")


def test_expert_layer():
    """As a serving program chains them: sorted, quantised to the sorted rows, grouped product,
    combined; against the same numbers in float64."""
    T, k, E, K, N = 70, 3, 6, 136, 90
    say("q8 expert layer")
    offsets, _, place, weights = routed(T, k, E, 9, 0.1)
    X, W, sw = rand((T, K), BF16, 1), bytes_of((E, N, K), 2, -127), positive((E, N), 3) / 64
    Q, s = sg.q8_quantize(X, place)
    Y = sg.q8_gemm(Q, s, W, sw, offsets, dtype=F32)
    out = sg.expert_combine(Y, place, weights)
    q, sx = quantize_reference(X)
    ends = offsets.tolist()
    ref, mag = torch.zeros((T, N), dtype=torch.float64, device="cuda"), 0
    mag = torch.zeros_like(ref)
    for t in range(T):
        for j in range(k):
            r = int(place[t, j])
            if r < 0:
                continue
            e = next(e for e in range(E) if ends[e] <= r < ends[e + 1])
            v = product(q[t:t + 1], sx[t:t + 1], W[e], sw[e])[0] * weights[t, j].double()
            ref[t] += v
            mag[t] += v.abs()
    check(out, ref, mag, k + 1 + 3, "layer")

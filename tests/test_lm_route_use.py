"""Rows sorted by expert and 8-bit products as a program uses them, on the GPU: an expert layer
in training and in serving, captured graphs, streams, repeated results, and operands past 2^31
elements."""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, check, rand  # noqa: E402
from .test_lm_use import bits  # noqa: E402
from .test_q8 import bytes_of, positive, product, quantize_reference  # noqa: E402

pytestmark = pytest.mark.gpu


def layer(dtype, T=60, k=3, H=96, F=72, E=5):
    g = torch.Generator().manual_seed(8)
    experts = torch.randint(-1, E, (T, k), generator=g).cuda()
    weights = (torch.rand((T, k), generator=g) + 0.1).cuda()
    A, B = rand((E, H, F), dtype, 2, H ** -0.5), rand((E, H, F), dtype, 3, F ** -0.5)
    return rand((T, H), dtype, 1), experts, weights, A, B


def forward(X, experts, weights, A, B):
    offsets, order, place = sg.expert_sort(experts, len(A))
    rows = sg.expert_gather(X, place)
    hidden = sg.grouped_gemm(rows, A, offsets)
    out = sg.grouped_gemm(hidden, B, offsets, trans=True)
    return sg.expert_combine(out, place, weights), (offsets, order, place, rows, hidden, out)


def backward(dY, X, weights, A, B, kept):
    offsets, _, place, rows, hidden, out = kept
    dout, dweights = sg.expert_combine_backward(dY, out, place, weights)
    dhidden = sg.grouped_gemm(dout, B, offsets)
    dB = sg.grouped_wgrad(dout, hidden, offsets)
    drows = sg.grouped_gemm(dhidden, A, offsets, trans=True)
    dA = sg.grouped_wgrad(rows, dhidden, offsets)
    return sg.expert_combine(drows, place), dweights, dA, dB


def test_training_step_of_an_expert_layer():
    """Sort, gather, two products, combine and every gradient in fp32 against autograd in
    float64.  Every value passes at most five sums of at most 96 terms: within 6 * 96 * 2^-24
    = 2^-14.8 of the magnitudes it sums over, which stay below ten times the largest here."""
    say("expert layer in training")
    X, experts, weights, A, B = layer(F32)
    Y, kept = forward(X, experts, weights, A, B)
    dY = rand(Y.shape, F32, 4)
    got = backward(dY, X, weights, A, B, kept)
    leaves = [t.double().requires_grad_() for t in (X, weights, A, B)]
    x, w, a, b = leaves
    ref = []
    for t in range(len(X)):
        row = x.new_zeros(x.shape[1])
        for j in range(experts.shape[1]):
            e = int(experts[t, j])
            if e >= 0:
                row = row + w[t, j] * ((x[t] @ a[e]) @ b[e].t())
        ref.append(row)
    ref = torch.stack(ref)
    grads = torch.autograd.grad((ref * dY.double()).sum(), leaves)
    for out, want in zip((Y,) + got, (ref.detach(),) + grads):
        assert out.shape == want.shape
        assert (out.double() - want).abs().max() <= 10 * 2.0 ** -14.8 * want.abs().max()


def test_serving_step_of_an_expert_layer():
    """The layer's weights quantised, its rows quantised on their way, each stage against its
    definition on what the stage before it gave."""
    say("expert layer in serving")
    X, experts, weights, A, B = layer(BF16, T=40, H=128, F=144)
    up, down = A.transpose(1, 2).contiguous(), B  # N x K
    (qa, sa), (qb, sb) = sg.q8_quantize(up), sg.q8_quantize(down)
    for w, q, s in ((up, qa, sa), (down, qb, sb)):
        ref, scale = quantize_reference(w.flatten(0, 1))
        assert torch.equal(q.flatten(0, 1), ref) and torch.equal(s.flatten(), scale)
    offsets, _, place = sg.expert_sort(experts, len(A))
    ends = offsets.tolist()
    Q, s = sg.q8_quantize(X, place)
    hidden = sg.q8_gemm(Q, s, qa, sa, offsets)
    Qh, sh = sg.q8_quantize(hidden)
    assert torch.equal(Qh, quantize_reference(hidden)[0])
    out = sg.q8_gemm(Qh, sh, qb, sb, offsets)
    assert torch.equal(out, sg.q8_matvec(hidden, qb, sb, offsets=offsets))
    for x, sx, w, sw, y in ((Q, s, qa, sa, hidden), (Qh, sh, qb, sb, out)):
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            ref = product(x[a:b], sx[a:b], w[e], sw[e])
            check(y[a:b], ref, ref.abs(), 3, "expert %d" % e)
        assert (y[ends[-1]:] == 0).all()
    Y = sg.expert_combine(out, place, weights)
    held = place >= 0
    terms = torch.where(held[..., None], out[place.clamp(min=0).long()].double() * weights.double()[..., None], 0.0)
    check(Y, terms.sum(1), terms.abs().sum(1), experts.shape[1] + 1, "combined")


def everything(X, experts, weights, A, B, dY, qa, sa, W, sw):
    """A training step, a serving step and a single token's product."""
    Y, kept = forward(X, experts, weights, A, B)
    grads = backward(dY, X, weights, A, B, kept)
    offsets, _, place = kept[:3]
    Q, s = sg.q8_quantize(X, place)
    hidden = sg.q8_gemm(Q, s, qa, sa, offsets, dtype=X.dtype)
    return (Y,) + grads + (kept[1], place, offsets, Q, s, hidden, sg.q8_matvec(X, qa[0], sa[0]),
                           sg.q8_matvec(X[:2], W, sw), sg.q8_gemm(Q[:, :W.shape[1]], s, W, sw, dtype=X.dtype))


def program(dtype, T=60, k=3):
    X, experts, weights, A, B = layer(dtype, T, k)
    return (X, experts, weights, A, B, rand(X.shape, dtype, 4), bytes_of((5, 72, 96), 5), positive((5, 72), 6) / 99,
            bytes_of((200, 96), 7), positive((200,), 8))


def raw(ts):
    return [t.contiguous().view(torch.uint8).clone() for t in ts]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k", [(60, 3), (9000, 2)])
def test_graphs(dtype, T, k):
    """Captured steps replayed on new inputs, with eager work between them, give the eager bits;
    two graphs keep what they allocate (the long sort's counts) apart."""
    say("route graphs", dtype, T, k)
    args = program(dtype, T, k)
    X, experts, weights = args[:3]
    everything(*args)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(*args))
        graphs.append(g)
    for n in range(4):
        X.copy_(rand(X.shape, dtype, 20 + n))
        experts.copy_(torch.randint(-1, 5, experts.shape, device="cuda"))
        weights.uniform_()
        want = raw(everything(*args))
        for g in graphs:
            g.replay()
        everything(*args)
        torch.cuda.synchronize()
        for o in outs:
            for got, ref in zip(raw(o), want):
                assert torch.equal(got, ref)


def test_streams():
    """Side streams, by argument and as the current one, several at once: the main stream's bits."""
    say("route streams")
    args = program(BF16)
    X, experts, weights, A, B, dY, qa, sa, W, sw = args
    want = raw(everything(*args))
    offsets, _, place = sg.expert_sort(experts, 5)
    Q, s = sg.q8_quantize(X, place)
    one = raw((offsets, place, sg.expert_gather(X, place, weights), sg.expert_combine(dY, place * 0, weights),
               *sg.expert_combine_backward(dY, X, place % 7, weights, need_dR=False)[1:], Q, s,
               sg.q8_gemm(Q, s, qa, sa, offsets), sg.q8_matvec(X, W, sw)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(everything(*args))
    side = []
    for st in streams:
        o, _, p = sg.expert_sort(experts, 5, stream=st)
        q, z = sg.q8_quantize(X, p, stream=st)
        side.append((o, p, sg.expert_gather(X, p, weights, stream=st),
                     sg.expert_combine(dY, place * 0, weights, stream=st),
                     sg.expert_combine_backward(dY, X, place % 7, weights, need_dR=False, stream=st)[1], q, z,
                     sg.q8_gemm(q, z, qa, sa, o, stream=st), sg.q8_matvec(X, W, sw, stream=st)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(raw(o), want))
    for o in side:
        assert all(torch.equal(a, b) for a, b in zip(raw(o), one))


def test_results_repeat():
    say("route repeats")
    args = program(F32, 5000, 3)
    first = raw(everything(*args))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(raw(everything(*args)), first))


@pytest.fixture
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.slow
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_past_32_bits(dtype, release):
    """Experts' rows, and tokens, more than 2^31 elements into their tensors."""
    T, k, H, E = (1 << 20) + 700, 2, 1040, 3
    assert T * H < 1 << 31 < T * k * H
    say("rows past 2^31 elements", dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    experts = torch.randint(0, E, (T, k), generator=g, device="cuda")
    offsets, order, place = sg.expert_sort(experts, E)
    key = experts.flatten()
    assert torch.equal(order.long(), torch.sort(key, stable=True).indices)
    weights = torch.rand((T, k), generator=g, device="cuda")
    X = rand((T, H), dtype, 2)
    R = sg.expert_gather(X, place)
    at = torch.cat([torch.arange(0, T * k, 4099, device="cuda"), torch.arange(T * k - 300, T * k, device="cuda")])
    assert torch.equal(R[at], X[order[at].long() // k])
    tokens = torch.cat([torch.arange(0, T, 4099, device="cuda"), torch.arange(T - 300, T, device="cuda")])
    out = sg.expert_combine(R, place, weights)
    x, w = X[tokens].double(), weights[tokens].double()
    check(out[tokens], x * w.sum(1)[:, None], x.abs() * w.sum(1)[:, None], k + 1, "combine")
    out.copy_(X)
    dR, dw = sg.expert_combine_backward(out, R, place, weights)
    slot = order[at].long()
    ref = X[slot // k].double() * weights.flatten()[slot].double()[:, None]
    check(dR[at], ref, ref.abs(), 1, "dR")
    dots = (x * x).sum(1)[:, None].expand(-1, k)
    check(dw[tokens], dots, dots, H + 1, "dweights")
    del dR, R, out
    Q, s = sg.q8_quantize(X, place)
    q, sx = quantize_reference(X[slot // k])
    assert torch.equal(Q[at], q) and torch.equal(s[at], sx)


@pytest.mark.slow
def test_8_bit_products_past_32_bits(release):
    """Weights, rows and results more than 2^31 elements into their tensors, one group's and many
    groups', for few rows and many."""
    say("8-bit products past 2^31")
    N, K = (1 << 19) + 300, 4112
    W, sw = torch.zeros((N, K), dtype=torch.int8, device="cuda"), positive((N,), 1)
    assert W.numel() > 1 << 31
    W[-400:] = bytes_of((400, K), 2)
    X = rand((20, K), BF16, 3)
    Q, s = sg.q8_quantize(X)
    ref = product(Q, s, W[-400:], sw[-400:])
    for Y in (sg.q8_gemm(Q, s, W, sw), sg.q8_gemm(Q[:7], s[:7], W, sw), sg.q8_matvec(X[:3], W, sw)):
        check(Y[:, -400:], ref[:len(Y)], ref[:len(Y)].abs(), 3, "one group")
        assert not Y[:, :-400].any()
    del W
    E, N = 600, 900
    W, sw = torch.zeros((E, N, K), dtype=torch.int8, device="cuda"), positive((E, N), 1)
    assert W.numel() > 1 << 31
    W[-1] = bytes_of((N, K), 2)
    for rows in (5, 3000):
        X = rand((rows, K), BF16, 3)
        Q, s = sg.q8_quantize(X)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = rows
        ref = product(Q, s, W[-1], sw[-1])
        check(sg.q8_gemm(Q, s, W, sw, off), ref, ref.abs(), 3, "many groups")
        if rows == 5:
            check(sg.q8_matvec(X, W, sw, offsets=off), ref, ref.abs(), 3, "many groups, few rows")
    del W, X, Q
    rows, K, N = (1 << 20) + 900, 2064, 2064
    Q = torch.zeros((rows, K), dtype=torch.int8, device="cuda")
    Q[-500:] = bytes_of((500, K), 4)
    W, sw, s = bytes_of((N, K), 5), positive((N,), 6), positive((rows,), 7)
    Y = sg.q8_gemm(Q, s, W, sw)
    assert Q.numel() > 1 << 31 and Y.numel() > 1 << 31
    ref = product(Q[-500:], s[-500:], W, sw)
    check(Y[-500:], ref, ref.abs(), 3, "rows")
    assert not Y[:-500].any()


@pytest.mark.slow
def test_more_rows_than_workgroups(release):
    """Past 2^24 workgroups of a few rows each, a workgroup takes several turns."""
    T = (1 << 26) + 37
    say("many rows")
    place = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, 1)
    X = torch.zeros((T, 2), dtype=BF16, device="cuda")
    X[-1], X[0] = torch.tensor([3.0, -1.5], device="cuda"), torch.tensor([0.5, 2.0], device="cuda")
    R = sg.expert_gather(X, place)
    assert torch.equal(R, X.flip(0))
    assert torch.equal(sg.expert_combine(R, place), X)
    dR, dw = sg.expert_combine_backward(X, R, place)
    assert torch.equal(dR, R) and dw[0].item() == 4.25 and dw[-1].item() == 11.25 and not dw[1:-1].any()
    Q, s = sg.q8_quantize(X)
    assert Q[-1].tolist() == [127, -64] and Q[0].tolist() == [32, 127] and not Q[1:-1].any()
    assert s[-1] == torch.tensor(3.0) * torch.tensor(1 / 127) and not s[1:-1].any()

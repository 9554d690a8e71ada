"""Rows sorted by expert, and back, on the GPU: the sort against counting on the host, the
copies and sums against their definitions in float64.

Tolerances.  A product of a weight and a value is rounded to fp32 once (2^-24 of itself) and a
bf16 result once more (half a step, 2^-8 of itself).  A sum of n fp32 products in any order
is off by at most (n + 1) 2^-24 times the sum of their magnitudes.
"""
import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import check, padded, rand  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def sort_reference(ids, E):
    """offsets, order, place of a list of experts' numbers, by Python's stable sort."""
    key = [e if 0 <= e < E else E for e in ids]
    order = sorted(range(len(key)), key=lambda s: key[s])
    place = [0] * len(key)
    for r, s in enumerate(order):
        place[s] = r if key[s] < E else -2 - r
    return [sum(x < e for x in key) for e in range(E + 1)], order, place


def choices(T, k, E, seed, outside=0.1):
    """Random choices, some outside [0, E) on either side."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, max(E, 1), (T, k), generator=g)
    out = torch.rand((T, k), generator=g) < (outside if E else 2.0)
    far = torch.tensor([-1, E, -(2 ** 62), 2 ** 32, 2 ** 62])[torch.randint(0, 5, (T, k), generator=g)]
    return torch.where(out, far, ids)


def assert_sorted(ids, E, got):
    offsets, order, place = got
    ref = sort_reference(ids.flatten().tolist(), E)
    assert offsets.tolist() == ref[0] and order.tolist() == ref[1]
    assert place.shape == ids.shape and place.flatten().tolist() == ref[2]


# One workgroup's chunk is 1024 slots or 2048 (half of that above 2048 experts); up to 16384 go in
# one launch.
@pytest.mark.parametrize("T,k", [(0, 2), (1, 0), (1, 1), (1, 7), (63, 1), (64, 1), (65, 3), (1024, 2),
                                 (2049, 1), (2731, 6), (5462, 3), (21000, 1)])
@pytest.mark.parametrize("E", [0, 1, 2, 7, 64, 257, 1024, 2048, 2049, 4096])
def test_sort(T, k, E):
    say("sort", T, k, E)
    ids = choices(T, k, E, T + 31 * k + E)
    assert_sorted(ids, E, sg.expert_sort(ids.cuda(), E))


@pytest.mark.parametrize("ids", ["one expert", "all dropped", "descending", "last only"])
def test_sort_of_uneven_choices(ids):
    T, E = 5000, 96
    t = {"one expert": torch.full((T, 1), 17), "all dropped": torch.full((T, 1), -5),
         "descending": (T - 1 - torch.arange(T)).view(T, 1) % E,
         "last only": torch.where(torch.arange(T) == T - 1, 0, E - 1).view(T, 1)}[ids]
    say("sort", ids)
    assert_sorted(t, E, sg.expert_sort(t.cuda(), E))


def test_sort_of_many_slots_takes_long_segments():
    """Past 256 chunks a segment is several of them."""
    for n, E in [(300001, 40), (256 * 2048 + 5, 40), (3 * 256 * 1024 + 77, 3000)]:
        say("sort", n, E)
        ids = torch.randint(-3, E + 3, (n, 1), generator=torch.Generator().manual_seed(n)).cuda()
        offsets, order, place = sg.expert_sort(ids, E)
        key = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
        ref = torch.sort(key, stable=True).indices
        assert torch.equal(order.long(), ref)
        row = torch.empty_like(ref)
        row[ref] = torch.arange(n, device="cuda")
        assert torch.equal(place.flatten().long(), torch.where(key < E, row, -2 - row))
        assert torch.equal(offsets.long(), torch.searchsorted(key[ref], torch.arange(E + 1, device="cuda")))


def routed(T, k, E, seed, outside=0.1):
    ids = choices(T, k, E, seed, outside).cuda()
    offsets, order, place = sg.expert_sort(ids, E)
    g = torch.Generator(device="cuda").manual_seed(seed)
    weights = torch.rand((T, k), generator=g, device="cuda") * 2 - 0.5
    return offsets, order.long(), place, weights


SHAPES = [(1, 1, 1), (1, 8, 64), (5, 3, 1), (33, 2, 7), (70, 9, 520), (17, 8, 1001), (6, 4, 2048), (3, 1, 5000)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_gather(dtype, T, k, H, pad, shift):
    say("gather", dtype, T, k, H, pad, shift)
    _, order, place, weights = routed(T, k, 5, T + H)
    held = (place.flatten()[order] >= 0)[:, None]
    X0 = rand((T, H), dtype, 1)
    X = padded(X0, pad, shift)
    rows, w = X0[order // k], weights.flatten()[order, None]
    out = sg.expert_gather(X, place)
    assert torch.equal(out, torch.where(held, rows, torch.zeros_like(rows)))
    ref = rows.double() * w.double() * held
    check(sg.expert_gather(X, place, weights), ref, ref.abs(), 1, "weighted")
    # Into rows of a larger buffer: what no choice has stays.
    old = rand((T * k + 3, H), dtype, 2)
    into = padded(old, pad, shift)
    base = into._base.clone()
    assert sg.expert_gather(X, place, out=into) is into
    assert torch.equal(into[:T * k], torch.where(held, rows, old[:T * k])) and torch.equal(into[T * k:], old[T * k:])
    into.copy_(old)
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(into._base.view(bits), base.view(bits))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_combine(dtype, T, k, H, pad, shift):
    say("combine", dtype, T, k, H, pad, shift)
    _, order, place, weights = routed(T, k, 5, T + H, 0.3)
    held = place >= 0
    R0 = rand((T * k, H), dtype, 1)
    # What no choice has is never read.
    R0[torch.ones(T * k, dtype=torch.bool, device="cuda").index_fill(0, place[held].long(), False)] = float("nan")
    weights = torch.where(held, weights, float("nan"))
    R = padded(R0, pad, shift)
    rows = torch.where(held[..., None], R0[place.clamp(min=0).long()], torch.zeros_like(R0[:1])).double()
    for w in (None, weights):
        terms = rows * (1.0 if w is None else torch.where(held, w, 0.0).double()[..., None])
        check(sg.expert_combine(R, place, w), terms.sum(1), terms.abs().sum(1), k + 1, "combine")
        old = rand((T, H), dtype, 2)
        out = padded(old, pad, shift)
        base = out._base.clone()
        assert sg.expert_combine(R, place, w, out, beta=-0.5) is out
        check(out, terms.sum(1) - 0.5 * old.double(), terms.abs().sum(1) + 0.5 * old.double().abs(), k + 2, "beta")
        out.copy_(old)
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(out._base.view(bits), base.view(bits))


def test_tokens_without_a_row_get_zeros():
    say("combine without rows")
    place = torch.tensor([[-1, -2], [1, -5], [-1, -1]], dtype=torch.int32, device="cuda")
    R = torch.tensor([[float("nan")], [3.0], [float("inf")], [float("nan")]], device="cuda")
    out = torch.full((3, 1), float("nan"), device="cuda")
    assert sg.expert_combine(R, place, out=out).flatten().tolist() == [0.0, 3.0, 0.0]
    assert sg.expert_combine(R, place.new_empty(3, 0)).flatten().tolist() == [0.0, 0.0, 0.0]
    assert sg.expert_combine(R[:0], place).flatten().tolist() == [0.0, 0.0, 0.0]
    dR, dw = sg.expert_combine_backward(out, R[:0], place)
    assert dR.shape == (0, 1) and dw.tolist() == [[0.0, 0.0]] * 3


def test_places_outside_the_rows_are_left_out():
    say("places outside")
    top, low = 2 ** 31 - 1, -2 ** 31
    place = torch.tensor([[0, 4, top], [low, -7, -1]], dtype=torch.int32, device="cuda")
    X = torch.ones(2, 8, device="cuda")
    R = torch.full((4, 8), 5.0, device="cuda")
    sg.expert_gather(X, place, out=R)
    assert R[:, 0].tolist() == [1.0, 5.0, 5.0, 5.0]
    assert sg.expert_combine(R, place)[:, 0].tolist() == [1.0, 0.0]
    dR, dw = sg.expert_combine_backward(X, R, place, dR=R.clone())
    assert dR[:, 0].tolist() == [1.0, 5.0, 5.0, 5.0] and dw.tolist() == [[8.0, 0.0, 0.0], [0.0, 0.0, 0.0]]
    Q, scales = sg.q8_quantize(X, torch.tensor([[9], [0]], dtype=torch.int32, device="cuda"))
    assert Q[0].tolist() == [127] * 8 and scales[0] * 127 == 1.0


# One, two and four waves a token (by H), four and eight choices at a time (by k).
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,H", SHAPES + [(4097, 3, 40), (5000, 9, 700), (40, 5, 900), (20, 2, 1000), (20, 3, 1000), (20, 2, 400),
                                            (20, 3, 400)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_combine_backward(dtype, T, k, H, pad, shift):
    say("combine backward", dtype, T, k, H, pad, shift)
    _, order, place, weights = routed(T, k, 5, T + H, 0.2)
    held = place >= 0
    R0 = rand((T * k, H), dtype, 1)
    R0[torch.ones(T * k, dtype=torch.bool, device="cuda").index_fill(0, place[held].long(), False)] = float("nan")
    weights = torch.where(held, weights, float("nan"))
    R, d0 = padded(R0, pad, shift), rand((T, H), dtype, 2)
    dout = padded(d0, pad, shift)
    rows = torch.where(held[..., None], R0[place.clamp(min=0).long()], torch.zeros_like(R0[:1])).double()
    dots = rows * d0.double()[:, None]
    for w in (None, weights):
        ref = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        terms = d0.double()[:, None] * (1.0 if w is None else w.double()[..., None])
        ref[place[held].long()] = terms.expand(T, k, H)[held]
        dR, dw = sg.expert_combine_backward(dout, R, place, w)
        check(dR, ref, ref.abs(), 1, "dR")
        check(dw, dots.sum(2), dots.abs().sum(2), H + 1, "dweights")
        assert (dw[~held] == 0).all()
        old = rand((T * k, H), dtype, 3)
        into = padded(old, pad, shift)
        given, none = sg.expert_combine_backward(dout, R, place, w, into, need_dweights=False)
        assert given is into and none is None
        mask = (place.flatten()[order] >= 0)[:, None]
        assert torch.equal(into, torch.where(mask, dR, old))
        none, dw2 = sg.expert_combine_backward(dout, R, place, w, need_dR=False)
        assert none is None and torch.equal(dw, dw2)


def test_gradients_against_differences():
    """Combine after gather as one function of the tokens and both weights: its gradients by
    the calls that the documentation names, against central differences in 64 bits."""
    T, k, H, E = 6, 3, 10, 4
    say("gradients against differences")
    _, _, place, w_out = routed(T, k, E, 3, 0.2)
    w_in = rand((T, k), F32, 4)
    X, dout = rand((T, H), F32, 5), rand((T, H), F32, 6)
    rows = sg.expert_gather(X, place, w_in)
    dR, dw_out = sg.expert_combine_backward(dout, rows, place, w_out)
    dX = sg.expert_combine(dR, place, w_in)
    dw_in = sg.expert_combine_backward(X, dR, place, need_dR=False)[1]
    held = (place >= 0).double()

    def value(X, w_in, w_out):
        return ((X[:, None] * (w_in * w_out * held)[..., None]).sum(1) * dout.double()).sum()
    args = [X.double(), w_in.double(), w_out.double()]
    for i, got in enumerate((dX, dw_in, dw_out)):
        for at in range(0, args[i].numel(), 5):
            h = 2.0 ** -10
            ends = []
            for sign in (1, -1):
                moved = [a.clone() for a in args]
                moved[i].view(-1)[at] += sign * h
                ends.append(value(*moved))
            # The function is linear in each argument: the difference is exact but for its
            # own rounding, and the fp32 sums' is some 30 steps of values around one.
            assert abs((ends[0] - ends[1]) / (2 * h) - got.view(-1)[at]) < 1e-4

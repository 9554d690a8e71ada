"""Rows sorted by expert and 8-bit products on streams that wait for what their operands were made
on, and from several host threads at once, on the GPU."""
import threading

import pytest

torch = pytest.importorskip("torch")

import fp32_gemm_04_amd as sg  # noqa: E402

from .gpu_helpers import say  # noqa: E402
from .test_lm_products import BF16, F32, rand  # noqa: E402
from .test_lm_route_use import raw  # noqa: E402
from .test_q8 import bytes_of, positive  # noqa: E402

pytestmark = pytest.mark.gpu


def operands(dtype, T=300, k=3, E=5, K=96, N=72):
    g = torch.Generator().manual_seed(6)
    experts = torch.randint(-1, E, (T, k), generator=g).cuda()
    weights = (torch.rand((T, k), generator=g) + 0.1).cuda()
    return experts, weights, rand((T, K), dtype, 1), bytes_of((E, N, K), 2), positive((E, N), 3)


def calls(experts, weights, X, W, sw, stream=None):
    """Every call, with operands that come from the calls before it; places that others share."""
    E = len(W)
    offsets, order, place = sg.expert_sort(experts, E, stream=stream)
    rows = sg.expert_gather(X, place, weights, stream=stream)
    back = sg.expert_combine(rows, place, weights, stream=stream)
    dR, dw = sg.expert_combine_backward(X, rows, place, weights, stream=stream)
    Q, s = sg.q8_quantize(X, place, stream=stream)
    Y = sg.q8_gemm(Q, s, W, sw, offsets, dtype=F32, stream=stream)
    out = sg.expert_combine(Y, place, weights, stream=stream)
    few = sg.q8_matvec(X[:3], W[0], sw[0], stream=stream)
    groups = sg.q8_matvec(X[:7], W, sw, offsets=offsets, stream=stream)
    return offsets, order, place, rows, back, dR, dw, Q, s, Y, out, few, groups


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_operands_made_on_another_stream(dtype):
    """Shared and remapped places are made on the main stream, and each side stream waits for it."""
    say("route streams that wait", dtype)
    experts, weights, X, W, sw = operands(dtype)
    main = torch.cuda.current_stream()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for n, st in enumerate(streams):
        e = (experts + n) % 5  # made just before the side stream takes it
        shared = torch.full_like(experts, n).int()
        x = X * (n + 1)
        st.wait_stream(main)
        offsets, order, place = sg.expert_sort(e, 5, stream=st)
        Q, s = sg.q8_quantize(x, place, stream=st)
        got.append((offsets, order, place, Q, s, sg.q8_gemm(Q, s, W, sw, offsets, stream=st),
                    sg.expert_combine(x, shared, weights, stream=st),
                    sg.expert_combine_backward(x, x, shared, weights, need_dR=False, stream=st)[1]))
    torch.cuda.synchronize()
    for n, o in enumerate(got):
        e, shared, x = (experts + n) % 5, torch.full_like(experts, n).int(), X * (n + 1)
        offsets, order, place = sg.expert_sort(e, 5)
        Q, s = sg.q8_quantize(x, place)
        want = (offsets, order, place, Q, s, sg.q8_gemm(Q, s, W, sw, offsets), sg.expert_combine(x, shared, weights),
                sg.expert_combine_backward(x, x, shared, weights, need_dR=False)[1])
        assert all(torch.equal(a, b) for a, b in zip(raw(o), raw(want)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_threads(dtype):
    """Three host threads, each on a stream of its own, ten times over: the main thread's bits."""
    say("route threads", dtype)
    args = operands(dtype)
    want = raw(calls(*args))
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(10):
                    out = calls(*args)
                    st.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(raw(out), want)):
                        wrong.append("bits")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))
    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]

"""Further language-model operators of libsgemm as cases to measure: tokens on
their way to experts and back, and products in 8-bit integers.

  dispatch      each token's expert numbers to rows sorted by expert (offsets,
                order, places), and the tokens' values copied to those rows
  combine       experts' output rows back to tokens, weighted and summed
  combine_step  the same with its gradients by the rows and the weights
  q8            tokens quantised to 8 bits with a scale each, times 8-bit weights
                with a scale for each output channel
  q8_experts    a serving expert layer's product: sorted, quantised straight to the
                sorted rows, multiplied by each expert's 8-bit weights, combined

``own`` true: the library's calls; false: elementary torch operations in 32 bits
(the quotients that are rounded to 8 bits in 64).
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # A few tokens in flight while serving, eight experts each.
        {"name": "dispatch_tokens_bf16", "kind": "dispatch", "type": "bf16", "T": 16, "k": 8, "E": 64,
         "H": 2048, "weighted": False},
        # One long prompt, two experts a token.
        {"name": "dispatch_prompt_bf16", "kind": "dispatch", "type": "bf16", "T": 8192, "k": 2,
         "E": 32, "H": 4096, "weighted": False},
        # A training batch over many small experts.
        {"name": "dispatch_batch_bf16", "kind": "dispatch", "type": "bf16", "T": 32768, "k": 8,
         "E": 256, "H": 1024, "weighted": False},
        # Single precision, weights applied on the way in, nothing a multiple of a vector.
        {"name": "dispatch_odd_f32", "kind": "dispatch", "type": "f32", "T": 4099, "k": 3, "E": 33,
         "H": 1001, "weighted": True},
        # The way back for a few tokens.
        {"name": "combine_tokens_bf16", "kind": "combine", "type": "bf16", "T": 24, "k": 8, "E": 64,
         "H": 2048},
        # A training step's way back and its gradients.
        {"name": "combine_step_bf16", "kind": "combine_step", "type": "bf16", "T": 16384, "k": 4,
         "E": 64, "H": 2048},
        # The same in single precision with odd sizes.
        {"name": "combine_step_odd_f32", "kind": "combine_step", "type": "f32", "T": 1500, "k": 5,
         "E": 24, "H": 777},
        # One token through a square layer: the smallest call of a serving loop.
        {"name": "q8_token_bf16", "kind": "q8", "type": "bf16", "T": 1, "K": 4096, "N": 4096},
        # A few sequences' tokens through a wide layer in single precision.
        {"name": "q8_rows_f32", "kind": "q8", "type": "f32", "T": 12, "K": 8192, "N": 28001},
        # A prompt through a wide layer.
        {"name": "q8_prompt_bf16", "kind": "q8", "type": "bf16", "T": 8192, "K": 4096, "N": 14336},
        # A short prompt in single precision, no size a multiple of a tile.
        {"name": "q8_odd_f32", "kind": "q8", "type": "f32", "T": 1023, "K": 1000, "N": 4999},
        # A prompt through the experts of one layer, held in 8 bits.
        {"name": "q8_experts_bf16", "kind": "q8_experts", "type": "bf16", "T": 4096, "k": 2, "E": 32,
         "K": 2048, "N": 1536},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["dispatch", "dispatch", "combine", "combine_step", "q8", "q8", "q8_experts"])
    t = rng.choice(["f32", "bf16"])
    step = rng.choice([1, 2, 8, 64])  # how round the sizes are

    def size(low, high):
        return max(step, _log(rng, low, high) // step * step)

    if kind == "q8":
        return {"kind": kind, "type": t, "T": _log(rng, 1, 8192), "K": size(64, 4096),
                "N": size(64, 14336)}
    E, k = _log(rng, 1, 256), rng.choice([1, 2, 3, 4, 6, 8])
    if kind == "q8_experts":
        E = min(E, 64)
        return {"kind": kind, "type": t, "T": _log(rng, 1, 4096), "k": min(k, 2), "E": E,
                "K": size(64, 2048), "N": size(64, 2048)}
    case = {"kind": kind, "type": t, "T": _log(rng, 1, 8192), "k": k, "E": E, "H": size(16, 2048)}
    if kind == "dispatch":
        case["weighted"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _experts(gen, T, k, E):
    """Each token's experts: some are asked for more than others, and about one token in
    thirty-two is padding that goes to none."""
    taste = torch.rand((E,), generator=gen, device="cuda") * 2.0
    noise = torch.rand((T, E), generator=gen, device="cuda").clamp(min=1e-6)
    scores = taste - torch.log(-torch.log(noise.clamp(max=1 - 1e-6)))
    ids = scores.topk(min(k, E), dim=1).indices
    if k > E:  # more choices than experts: the same ones again
        ids = ids.repeat(1, -(-k // E))[:, :k]
    padding = torch.rand((T, 1), generator=gen, device="cuda") < 1.0 / 32
    return torch.where(padding, torch.full_like(ids, -1), ids).contiguous()


def _weights(gen, T, k):
    w = torch.rand((T, k), generator=gen, device="cuda") + 0.1
    return w / w.sum(1, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, t, T = case["kind"], TYPES[case["type"]], case["T"]
    s = {"case": case}
    if kind == "q8":
        K, N = case["K"], case["N"]
        s["X"] = _tokens(gen, T, K, t)
        s["Q"], s["scales"] = _q8_weights(gen, (N, K))
        return s
    k, E = case["k"], case["E"]
    s["experts"] = _experts(gen, T, k, E)
    if kind == "q8_experts":
        K, N = case["K"], case["N"]
        s["X"] = _tokens(gen, T, K, t)
        s["Q"], s["scales"] = _q8_weights(gen, (E, N, K))
        s["weights"] = _weights(gen, T, k)
        return s
    H = case["H"]
    if kind == "dispatch":
        s["X"] = _normal(gen, (T, H), 1.0, t)
        s["weights"] = _weights(gen, T, k) if case["weighted"] else None
        return s
    s["place"] = _plain_sort(s["experts"], E)[2]
    s["Y"] = _normal(gen, (T * k, H), 1.0, t)
    s["weights"] = _weights(gen, T, k)
    if kind == "combine_step":
        s["dout"] = _normal(gen, (T, H), 1.0, t)
    return s


def _tokens(gen, T, K, t):
    """Hidden values whose size differs from token to token, a few channels larger."""
    X = torch.randn((T, K), generator=gen, device="cuda")
    X *= torch.exp(torch.randn((T, 1), generator=gen, device="cuda"))
    X *= 1.0 + 7.0 * (torch.rand((K,), generator=gen, device="cuda") < 1.0 / 128)
    return X.to(t)


def _q8_weights(gen, shape):
    Q = torch.randn(shape, generator=gen, device="cuda").mul_(32.0).round_().clamp_(-127, 127)
    scales = (torch.rand(shape[:-1], generator=gen, device="cuda") + 0.5) / (32 * math.sqrt(shape[-1]))
    return Q.to(torch.int8), scales


# ------------------------------------------------------------- plain forms

def _plain_sort(experts, E):
    ids = experts.flatten()
    ids = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E))
    order = torch.sort(ids, stable=True).indices
    counts = (ids[:, None] == torch.arange(E, device=ids.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    row = torch.empty_like(order)
    row[order] = torch.arange(ids.numel(), device=ids.device)
    place = torch.where(ids < E, row, -2 - row)
    return offsets.int(), order.int(), place.int().reshape(experts.shape)


def _plain_gather(X, order, place, weights):
    k = place.shape[1]
    slots = order.long()
    rows = X[slots // k]
    if weights is not None:
        rows = rows.float() * weights.flatten()[slots, None]
    return torch.where((place.flatten()[slots] >= 0)[:, None], rows, torch.zeros_like(rows)).to(X.dtype)


def _plain_combine(Y, place, weights):
    held = (place >= 0).float()
    out = torch.zeros((place.shape[0], Y.shape[1]), device=Y.device)
    for j in range(place.shape[1]):
        out += Y[place[:, j].clamp(min=0).long()].float() * (weights[:, j] * held[:, j])[:, None]
    return out.to(Y.dtype)


def _plain_quantize(X):
    """Whole numbers as floats, and each row's scale."""
    scales = X.float().abs().amax(1) / 127.0
    Q = torch.round(X.double() / scales.double()[:, None]).nan_to_num_(0.0).clamp_(-127, 127)
    return Q.float(), scales


def _plain(s):
    case = s["case"]
    kind, t = case["kind"], TYPES[case["type"]]
    if kind == "dispatch":
        offsets, order, place = _plain_sort(s["experts"], case["E"])
        return {"offsets": offsets, "order": order, "place": place,
                "rows": _plain_gather(s["X"], order, place, s["weights"])}
    if kind == "combine":
        return _plain_combine(s["Y"], s["place"], s["weights"])
    if kind == "combine_step":
        place, Y, dout, w = s["place"], s["Y"], s["dout"].float(), s["weights"]
        dY, dw = torch.zeros(Y.shape, device=Y.device), torch.zeros_like(w)
        for j in range(place.shape[1]):
            held = (place[:, j] >= 0).float()
            rows = torch.where(place[:, j] >= 0, place[:, j], -2 - place[:, j]).long()
            dY[rows] = dout * (w[:, j] * held)[:, None]
            dw[:, j] = (dout * Y[rows].float()).sum(1) * held
        return {"out": _plain_combine(Y, place, w), "dY": dY.to(t), "dweights": dw}
    Q, scales = _plain_quantize(s["X"])
    if kind == "q8":
        return ((Q @ s["Q"].float().t()) * scales[:, None] * s["scales"]).to(t)
    offsets, order, place = _plain_sort(s["experts"], case["E"])
    slots, ends = order.long(), offsets.tolist()
    Qs, ss = Q[slots // case["k"]], scales[slots // case["k"]]
    Y = torch.zeros((slots.numel(), case["N"]), device="cuda")
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            Y[a:b] = (Qs[a:b] @ s["Q"][e].float().t()) * ss[a:b, None] * s["scales"][e]
    return _plain_combine(Y, place, s["weights"]).to(t)


def run(state):
    if not own:
        return _plain(state)
    import fp32_gemm_04_amd as sg
    s, case = state, state["case"]
    kind, t = case["kind"], TYPES[case["type"]]
    if kind == "dispatch":
        offsets, order, place = sg.expert_sort(s["experts"], case["E"])
        rows = sg.expert_gather(s["X"], place, s["weights"])
        return {"offsets": offsets, "order": order, "place": place, "rows": rows}
    if kind == "combine":
        return sg.expert_combine(s["Y"], s["place"], s["weights"])
    if kind == "combine_step":
        out = sg.expert_combine(s["Y"], s["place"], s["weights"])
        dY, dw = sg.expert_combine_backward(s["dout"], s["Y"], s["place"], s["weights"])
        return {"out": out, "dY": dY, "dweights": dw}
    if kind == "q8":
        if case["T"] <= 16:
            return sg.q8_matvec(s["X"], s["Q"], s["scales"])
        Q, scales = sg.q8_quantize(s["X"])
        return sg.q8_gemm(Q, scales, s["Q"], s["scales"], dtype=t)
    offsets, _, place = sg.expert_sort(s["experts"], case["E"])
    Q, scales = sg.q8_quantize(s["X"], place)
    # The experts' rows stay in 32 bits until their weighted sum, which alone is rounded to t.
    Y = sg.q8_gemm(Q, scales, s["Q"], s["scales"], offsets=offsets, dtype=torch.float32)
    return sg.expert_combine(Y, place, s["weights"]).to(t)


def work(case):
    b, T = SIZE[case["type"]], case["T"]
    if case["kind"] == "q8":
        K, N = case["K"], case["N"]
        return {"bytes": b * T * (K + N) + N * K + 4 * N, "flops": 2.0 * T * K * N}
    n = T * case["k"]
    if case["kind"] == "q8_experts":
        K, N, E = case["K"], case["N"], case["E"]
        used = min(E, n)  # about all experts of a long batch
        return {"bytes": b * T * (K + N) + used * (N * K + 4 * N) + 12 * n, "flops": 2.0 * n * K * N}
    H = case["H"]
    if case["kind"] == "dispatch":
        # The experts' numbers; offsets, order and places; tokens once, rows once.
        return {"bytes": 16 * n + b * (T + n) * H + (4 * n if case["weighted"] else 0),
                "flops": float(n * H) if case["weighted"] else 0.0}
    combine = {"bytes": 8 * n + b * (T + n) * H, "flops": 2.0 * n * H}
    if case["kind"] == "combine":
        return combine
    # The rows of Y once for both directions; dY and the weights' gradient written.
    return {"bytes": combine["bytes"] + b * (T + n) * H + 4 * n, "flops": 5.0 * n * H}


# ------------------------------------------------- the definition in 64 bits

def _exact_place(experts, E):
    """Row of every slot, by counting: slots of lower experts, and earlier ones of its own;
    slots of no expert come last."""
    ids = experts.flatten().cpu()
    lists = [[] for _ in range(E + 1)]
    for slot, e in enumerate(ids.tolist()):
        lists[e if 0 <= e < E else E].append(slot)
    order, ends = [], [0]
    for e in range(E + 1):
        order += lists[e]
        ends.append(len(order))
    place = torch.empty(ids.numel(), dtype=torch.int64)
    place[torch.tensor(order, dtype=torch.int64)] = torch.arange(len(order))
    place = torch.where((ids >= 0) & (ids < E), place, -2 - place)
    return (torch.tensor(ends[:-1], dtype=torch.int32, device="cuda"),
            torch.tensor(order, dtype=torch.int32, device="cuda"),
            place.int().reshape(experts.shape).cuda())


def _exact_combine(Y, place, weights):
    T, k = place.shape
    out = torch.zeros((T, Y.shape[1]), dtype=torch.float64, device="cuda")
    t, j = (place >= 0).nonzero(as_tuple=True)
    for a in range(0, t.numel(), 16384):
        ta, ja = t[a:a + 16384], j[a:a + 16384]
        out.index_add_(0, ta, Y[place[ta, ja].long()].double() * weights[ta, ja].double()[:, None])
    return out


def _exact_quantize(X):
    """Dequantised by nothing but its own scale: the whole numbers and the scales, the scale
    being the stored 32-bit one."""
    X = X.double()
    scales = (X.abs().max(dim=1).values / 127.0).float().double()
    safe = torch.where(scales > 0, scales, torch.ones_like(scales))
    whole = torch.floor(X / safe[:, None] + 0.5)
    tie = (X / safe[:, None] + 0.5) == whole
    whole = torch.where(tie & (whole.remainder(2) == 1), whole - 1, whole)
    return whole.clamp(-127, 127), scales


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "q8":
        Q, scales = _exact_quantize(s["X"])
        W = s["Q"].double() * s["scales"].double()[:, None]
        return (Q * scales[:, None]) @ W.t()
    if kind in ("combine", "combine_step"):
        Y, place, w = s["Y"], s["place"], s["weights"]
        out = _exact_combine(Y, place, w)
        if kind == "combine":
            return out
        dY = torch.zeros(Y.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(place.shape, dtype=torch.float64, device="cuda")
        for j in range(place.shape[1]):
            t = (place[:, j] >= 0).nonzero()[:, 0]
            at = place[t, j].long()
            d = s["dout"][t].double()
            dY[at] = d * w[t, j].double()[:, None]
            dw[t, j] = torch.einsum("th,th->t", d, Y[at].double())
        return {"out": out, "dY": dY, "dweights": dw}
    offsets, order, place = _exact_place(s["experts"], case["E"])
    if kind == "dispatch":
        rows = torch.zeros((order.numel(), case["H"]), dtype=torch.float64, device="cuda")
        t, j = (place >= 0).nonzero(as_tuple=True)
        for a in range(0, t.numel(), 16384):
            ta, ja = t[a:a + 16384], j[a:a + 16384]
            v = s["X"][ta].double()
            if s["weights"] is not None:
                v = v * s["weights"][ta, ja].double()[:, None]
            rows[place[ta, ja].long()] = v
        return {"offsets": offsets, "order": order, "place": place, "rows": rows}
    Q, scales = _exact_quantize(s["X"])
    X = Q * scales[:, None]
    out = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = (s["experts"] == e).nonzero(as_tuple=True)
        if t.numel():
            W = s["Q"][e].double() * s["scales"][e].double()[:, None]
            out.index_add_(0, t, (X[t] @ W.t()) * s["weights"][t, j].double()[:, None])
    return out

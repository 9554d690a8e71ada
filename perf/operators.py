"""The language-model products of libsgemm as cases to measure.

Three families, each in the library's form (``own`` true) and in a plain form
of elementary torch operations in 32 bits (``own`` false):

  experts   rows sorted by expert, each expert's rows times its own weights
            (forward), and the gradients of rows and weights (backward)
  xent      softmax cross entropy of an output layer's logits, from the hidden
            rows and the vocabulary's weights, alone or with both gradients
  q4        rows times weights held in 4 bits with a scale and an offset for
            each block of weights, for one set of weights or one per expert
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # A few tokens in flight while serving: every expert in use has one or two rows.
        {"name": "experts_tokens_bf16", "kind": "experts", "type": "bf16", "E": 32, "T": 24,
         "K": 2048, "N": 1408, "trans": True, "sizes": 1},
        # One sequence's prompt through the experts, weights stored input-major.
        {"name": "experts_prompt_bf16", "kind": "experts", "type": "bf16", "E": 64, "T": 8192,
         "K": 2048, "N": 1536, "trans": False, "sizes": 2},
        # Single precision with rows and columns that no tile divides, and rows that are
        # not 16-byte aligned.
        {"name": "experts_odd_f32", "kind": "experts", "type": "f32", "E": 8, "T": 4099,
         "K": 1000, "N": 1537, "trans": False, "sizes": 3},
        # A training step's backward pass of one expert layer.
        {"name": "experts_backward_bf16", "kind": "experts_backward", "type": "bf16", "E": 16,
         "T": 16384, "K": 2048, "N": 2048, "trans": False, "sizes": 4},
        # The same for a small layer in single precision, ragged everywhere.
        {"name": "experts_backward_f32", "kind": "experts_backward", "type": "f32", "E": 24,
         "T": 1500, "K": 520, "N": 772, "trans": True, "sizes": 5},
        # Scoring one short text: the loss alone.
        {"name": "xent_score_f32", "kind": "xent", "type": "f32", "T": 37, "H": 1024, "V": 32000},
        # A fine-tuning step on a short batch.
        {"name": "xent_step_short_bf16", "kind": "xent_step", "type": "bf16", "T": 384, "H": 1024,
         "V": 50021},
        # A training step of a large vocabulary's output layer.
        {"name": "xent_step_bf16", "kind": "xent_step", "type": "bf16", "T": 8192, "H": 2048,
         "V": 131072},
        # A training step in single precision, no size a multiple of a tile.
        {"name": "xent_step_odd_f32", "kind": "xent_step", "type": "f32", "T": 1023, "H": 1000,
         "V": 49999},
        # One token through a square layer: the smallest call of a serving loop.
        {"name": "q4_token_bf16", "kind": "q4", "type": "bf16", "E": 1, "T": 1, "K": 4096,
         "N": 4096, "block": 128, "zeros": True, "sizes": 0},
        # A few sequences' tokens through a wide layer in single precision.
        {"name": "q4_rows_f32", "kind": "q4", "type": "f32", "E": 1, "T": 12, "K": 8192,
         "N": 28001, "block": 32, "zeros": False, "sizes": 0},
        # Tokens spread over experts whose weights are held in 4 bits.
        {"name": "q4_experts_bf16", "kind": "q4", "type": "bf16", "E": 32, "T": 48, "K": 2048,
         "N": 5632, "block": 64, "zeros": True, "sizes": 6},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["experts", "experts", "experts_backward", "xent", "xent_step", "q4", "q4"])
    t = rng.choice(["f32", "bf16"])
    step = rng.choice([1, 2, 8, 64])  # how round the sizes are

    def size(low, high, by=None):
        by = by or step
        return max(by, _log(rng, low, high) // by * by)

    if kind in ("experts", "experts_backward"):
        E = _log(rng, 1, 64)
        most = 8192 if t == "bf16" else 4096
        return {"kind": kind, "type": t, "E": E, "T": _log(rng, 1, most), "K": size(64, 2048),
                "N": size(64, 2048), "trans": rng.random() < 0.5, "sizes": rng.randrange(1 << 20)}
    if kind in ("xent", "xent_step"):
        most = 4096 if t == "bf16" else 1024
        return {"kind": kind, "type": t, "T": _log(rng, 1, most), "H": size(64, 2048),
                "V": size(1000, 131072)}
    E = rng.choice([1, 1, 4, 8, 32])
    return {"kind": "q4", "type": t, "E": E, "T": _log(rng, 1, 64), "K": size(256, 8192, 2 * step),
            "N": size(64, 16384 if E == 1 else 4096), "block": rng.choice([32, 64, 128]),
            "zeros": rng.random() < 0.5, "sizes": rng.randrange(1 << 20)}


def _sizes(case):
    """Rows of each expert: uneven, about one expert in eight without any."""
    E, T = case["E"], case["T"]
    if E == 1:
        return [T]
    rng = random.Random(case["sizes"])
    weights = [0.0 if rng.random() < 0.125 else rng.uniform(0.5, 1.5) for _ in range(E)]
    if not any(weights):
        weights[rng.randrange(E)] = 1.0
    if T < 4 * E:
        counts = [0] * E
        for e in rng.choices(range(E), weights, k=T):
            counts[e] += 1
        return counts
    total, done, left, counts = sum(weights), 0.0, T, []
    for w in weights:
        done += w
        n = T - int(round(T * (1 - done / total))) - (T - left)
        counts.append(n)
        left -= n
    return counts


def _normal(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, t = case["kind"], TYPES[case["type"]]
    s = {"case": case}
    if kind in ("xent", "xent_step"):
        T, H, V = case["T"], case["H"], case["V"]
        s["X"] = _normal(gen, (T, H), 1.0, t)
        s["W"] = _normal(gen, (V, H), 2.0 / math.sqrt(H), t)
        targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
        # About one row in sixteen is padding and does not count.
        skip = torch.rand((T,), generator=gen, device="cuda") < 1.0 / 16
        s["targets"] = torch.where(skip, torch.full_like(targets, -100), targets)
        s["dloss"] = (torch.rand((T,), generator=gen, device="cuda") + 0.5) / T
        return s
    E, T, K, N = case["E"], case["T"], case["K"], case["N"]
    counts = _sizes(case)
    s["most"] = max(counts)
    ends = [0]
    for n in counts:
        ends.append(ends[-1] + n)
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["X"] = _normal(gen, (T, K), 1.0, t)
    if kind == "q4":
        block, G = case["block"], -(-K // case["block"])
        s["Q"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda",
                               dtype=torch.int32).to(torch.uint8)
        s["scales"] = ((torch.rand((E, N, G), generator=gen, device="cuda") + 0.5)
                       * (0.2 / math.sqrt(K))).to(t)
        s["zeros"] = (torch.randint(5, 11, (E, N, G), generator=gen, device="cuda",
                                    dtype=torch.int32).to(torch.uint8) if case["zeros"] else None)
        if E == 1:
            for k in ("Q", "scales", "zeros"):
                s[k] = s[k][0] if s[k] is not None else None
            s["offsets"] = None
        return s
    shape = (E, N, K) if case["trans"] else (E, K, N)
    s["W"] = _normal(gen, shape, 1.0 / math.sqrt(K), t)
    if kind == "experts":
        s["Y"] = torch.zeros((T, N), dtype=t, device="cuda")
    else:
        s["dY"] = _normal(gen, (T, N), 1.0, t)
        s["dX"] = torch.zeros((T, K), dtype=t, device="cuda")
        s["dW"] = torch.zeros(shape, dtype=t, device="cuda")
    return s


# ------------------------------------------------------------ plain forms

def _places(s, T):
    """Each row's expert and its place among that expert's rows, and the rows of every
    (expert, place) with the places that hold none marked."""
    offsets = s["offsets"].long()
    rows = torch.arange(T, device="cuda")
    expert = torch.bucketize(rows, offsets[1:], right=True)
    place = rows - offsets[expert]
    at = offsets[:-1, None] + torch.arange(s["most"], device="cuda")
    held = at < offsets[1:, None]
    return expert, place, at.clamp(max=T - 1), held


def _pad(rows, at, held):
    return rows.float()[at] * held[..., None]


def _q4_weights(s, case):
    Q, block = s["Q"], case["block"]
    q = torch.stack([Q & 15, Q >> 4], dim=-1).flatten(-2).float()
    scales = s["scales"].float().repeat_interleave(block, dim=-1)[..., :case["K"]]
    if s["zeros"] is None:
        return (q - 8.0) * scales
    return (q - s["zeros"].float().repeat_interleave(block, dim=-1)[..., :case["K"]]) * scales


def _plain_experts(X, W, s, case):
    T = case["T"]
    expert, place, at, held = _places(s, T)
    return torch.bmm(_pad(X, at, held), W)[expert, place]


def _plain(s):
    case = s["case"]
    kind, t = case["kind"], TYPES[case["type"]]
    if kind == "experts":
        W = s["W"].float()
        return _plain_experts(s["X"], W.transpose(1, 2) if case["trans"] else W, s, case).to(t)
    if kind == "experts_backward":
        W = s["W"].float()
        expert, place, at, held = _places(s, case["T"])
        Xp, dYp = _pad(s["X"], at, held), _pad(s["dY"], at, held)
        dX = torch.bmm(dYp, W if case["trans"] else W.transpose(1, 2))[expert, place]
        if case["trans"]:
            dW = torch.bmm(dYp.transpose(1, 2), Xp)
        else:
            dW = torch.bmm(Xp.transpose(1, 2), dYp)
        return {"dX": dX.to(t), "dW": dW.to(t)}
    if kind == "q4":
        W = _q4_weights(s, case)
        if case["E"] == 1:
            return (s["X"].float() @ W.t()).to(t)
        return _plain_experts(s["X"], W.transpose(1, 2), s, case).to(t)
    X, W, targets = s["X"].float(), s["W"].float(), s["targets"]
    counts = targets >= 0
    logits = X @ W.t()
    top = logits.amax(dim=1, keepdim=True)
    e = (logits - top).exp()
    total = e.sum(dim=1, keepdim=True)
    lse = (top + total.log())[:, 0]
    label = targets.clamp(min=0)
    loss = torch.where(counts, lse - logits.gather(1, label[:, None])[:, 0], torch.zeros_like(lse))
    if kind == "xent":
        return {"loss": loss, "lse": lse}
    g = torch.where(counts, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    d = e / total * g
    d.scatter_add_(1, label[:, None], -g)
    return {"loss": loss, "dX": (d @ W).to(t), "dW": (d.t() @ X).to(t)}


def run(state):
    if not own:
        return _plain(state)
    import fp32_gemm_04_amd as sg
    s, case = state, state["case"]
    kind = case["kind"]
    if kind == "experts":
        return sg.grouped_gemm(s["X"], s["W"], s["offsets"], s["Y"], trans=case["trans"])
    if kind == "experts_backward":
        sg.grouped_gemm(s["dY"], s["W"], s["offsets"], s["dX"], trans=not case["trans"])
        if case["trans"]:
            sg.grouped_wgrad(s["dY"], s["X"], s["offsets"], s["dW"])
        else:
            sg.grouped_wgrad(s["X"], s["dY"], s["offsets"], s["dW"])
        return {"dX": s["dX"], "dW": s["dW"]}
    if kind == "q4":
        return sg.q4_matvec(s["X"], s["Q"], s["scales"], s["zeros"], block=case["block"],
                            offsets=s["offsets"])
    loss, lse = sg.linear_cross_entropy(s["X"], s["W"], s["targets"])
    if kind == "xent":
        return {"loss": loss, "lse": lse}
    dX, dW = sg.linear_cross_entropy_backward(s["dloss"], s["X"], s["W"], s["targets"], lse)
    return {"loss": loss, "dX": dX, "dW": dW}


def work(case):
    b = SIZE[case["type"]]
    if case["kind"] in ("xent", "xent_step"):
        T, H, V = case["T"], case["H"], case["V"]
        if case["kind"] == "xent":
            return {"bytes": b * (T * H + V * H) + 16 * T, "flops": 2.0 * T * H * V}
        # The logits once and the two gradients.
        return {"bytes": 2 * b * (T * H + V * H) + 16 * T, "flops": 6.0 * T * H * V}
    E, T, K, N = case["E"], case["T"], case["K"], case["N"]
    used = sum(n > 0 for n in _sizes(case))
    if case["kind"] == "q4":
        G = -(-K // case["block"])
        w = used * N * (K // 2 + G * (b + (1 if case["zeros"] else 0)))
        return {"bytes": w + b * T * (K + N), "flops": 2.0 * T * K * N}
    if case["kind"] == "experts":
        return {"bytes": b * (used * K * N + T * (K + N)), "flops": 2.0 * T * K * N}
    # dX reads dY and the weights in use; dW reads X and dY and writes every expert's.
    return {"bytes": b * ((used + E) * K * N + 2 * T * (K + N)), "flops": 4.0 * T * K * N}


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    X = s["X"].double()
    if kind in ("xent", "xent_step"):
        W, T = s["W"].double(), case["T"]
        loss, lse = X.new_zeros(T), X.new_zeros(T)
        dX, dW = torch.zeros_like(X), torch.zeros_like(W)
        for a in range(0, T, 1024):
            z = X[a:a + 1024] @ W.t()
            y = s["targets"][a:a + 1024]
            m = z.max(1).values
            lse[a:a + 1024] = m + torch.log(torch.exp(z - m[:, None]).sum(1))
            p = torch.exp(z - lse[a:a + 1024, None])
            for_rows = (y >= 0).nonzero()[:, 0]
            loss[a + for_rows] = lse[a + for_rows] - z[for_rows, y[for_rows]]
            if kind == "xent_step":
                p[for_rows, y[for_rows]] -= 1.0
                weight = s["dloss"][a:a + 1024].double() * (y >= 0)
                p *= weight[:, None]
                dX[a:a + 1024] = p @ W
                dW += p.t() @ X[a:a + 1024]
        return {"loss": loss, "lse": lse} if kind == "xent" else {"loss": loss, "dX": dX, "dW": dW}
    counts = _sizes(case)
    if kind == "q4":
        Q = s["Q"].reshape(case["E"], case["N"], -1).to(torch.int64)
        q = torch.empty((case["E"], case["N"], case["K"]), dtype=torch.float64, device="cuda")
        q[..., 0::2] = (Q % 16).double()
        q[..., 1::2] = (Q // 16).double()
        of = torch.arange(case["K"], device="cuda") // case["block"]
        zeros = (s["zeros"].reshape(case["E"], case["N"], -1).double()[..., of]
                 if s["zeros"] is not None else 8.0)
        W = (q - zeros) * s["scales"].reshape(case["E"], case["N"], -1).double()[..., of]
        W = W.transpose(1, 2)
    else:
        W = s["W"].double()
        W = W.transpose(1, 2) if case["trans"] else W
    at = 0
    if kind != "experts_backward":
        Y = X.new_zeros((case["T"], case["N"]))
        for e, n in enumerate(counts):
            Y[at:at + n] = X[at:at + n] @ W[e]
            at += n
        return Y
    dY = s["dY"].double()
    dX, dW = torch.zeros_like(X), torch.zeros_like(W)
    for e, n in enumerate(counts):
        dX[at:at + n] = dY[at:at + n] @ W[e].t()
        dW[e] = X[at:at + n].t() @ dY[at:at + n]
        at += n
    return {"dX": dX, "dW": dW.transpose(1, 2).contiguous() if case["trans"] else dW}

"""Cases of the 4-bit weight operators: the encoder, the skinny product and the mixture-of-experts layer.

A weight is held as 4-bit codes q in 0..15 with one 16-bit scale s and one zero point z for each group of 32, 64 or
128 neighbours along K: w = s * (q - z), z = 8 where no zero points are kept.

  encode  a dense fp16 or bf16 weight to that form and back to dense
  matmul  C[N, M] = B[N, K] x A[M, K]^T with A in that form, N = 1 .. 256 tokens
  moe     router, top-k, gated experts in that form and their weighted sum, for 1 .. 64 tokens

With `own` false, `run` computes them from elementary torch operations in fp32 (router logits in fp64: their order
decides which experts run); with `own` true it calls the package.
"""
import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
LARGEST_WEIGHT = 49152 * 12288          # values of the largest single matrix below
LARGEST_EXPERTS = 64 * 3 * 4096 * 2048  # values of the largest stack of experts below


def listed():
    def encode(name, M, K, dtype, group, symmetric):
        return {"name": name, "op": "encode", "M": M, "K": K, "dtype": dtype, "group": group, "symmetric": symmetric}

    def matmul(name, M, K, N, dtype, group, symmetric):
        return {"name": name, "op": "matmul", "M": M, "K": K, "N": N, "dtype": dtype, "group": group,
                "symmetric": symmetric}

    def moe(name, T, E, k, H, F, dtype, group, symmetric, renormalize=True, activation="silu"):
        return {"name": name, "op": "moe", "T": T, "E": E, "k": k, "H": H, "F": F, "dtype": dtype, "group": group,
                "symmetric": symmetric, "renormalize": renormalize, "activation": activation}

    return [
        # a small projection quantised while a model is loaded
        encode("encode-4096sq-bf16", 4096, 4096, "bf16", 128, False),
        # the QKV weight of the OPT-175B-shaped layer
        encode("encode-36864x12288-fp16", 36864, 12288, "fp16", 64, True),
        # one token through the LLaMA-7B-shaped output projection: the latency of a single small product
        matmul("matmul-n1-4096sq-bf16", 4096, 4096, 1, "bf16", 128, True),
        # one token through the first MLP weight of the OPT-175B-shaped layer: the longest single-token product
        matmul("matmul-n1-49152x12288-fp16", 49152, 12288, 1, "fp16", 128, False),
        # a few tokens (speculative decoding, a small batch) through the gate of the LLaMA-7B-shaped MLP
        matmul("matmul-n5-11008x4096-bf16", 11008, 4096, 5, "bf16", 64, False),
        # odd everything: rows, columns (unaligned activations) and tokens, finest groups
        matmul("matmul-n17-4099x5003-fp16", 4099, 5003, 17, "fp16", 32, False),
        # a serving batch on the square weight of the stress sweep
        matmul("matmul-n64-12288sq-bf16", 12288, 12288, 64, "bf16", 128, True),
        # the widest batch on the second MLP weight of the OPT-66B-shaped layer (long K)
        matmul("matmul-n256-9216x36864-fp16", 9216, 36864, 256, "fp16", 64, True),
        # one token, many small experts: latency of the whole layer
        moe("moe-t1-e128k8-2048x768-bf16", 1, 128, 8, 2048, 768, "bf16", 128, True),
        # four tokens, few large experts with the LLaMA-7B-shaped MLP
        moe("moe-t4-e8k2-4096x11008-fp16", 4, 8, 2, 4096, 11008, "fp16", 64, False),
        # an odd number of tokens over experts of a width that ends inside a tile, weights left as the softmax gave them
        moe("moe-t33-e60k6-2056x1416-bf16", 33, 60, 6, 2056, 1416, "bf16", 32, False, False, "gelu"),
        # the most tokens: every expert runs
        moe("moe-t64-e64k8-4096x2048-bf16", 64, 64, 8, 4096, 2048, "bf16", 128, True),
    ]


def _spread(rng, low, high):
    """A whole number of low .. high, even over its logarithm; one in three is made odd."""
    v = int(round(low * (high / low) ** rng.random()))
    return min(high, max(low, v | 1 if rng.random() < 0.34 else v - v % 8 if v >= 64 else v))


def draw(rng):
    op = rng.choice(["encode", "matmul", "matmul", "moe", "moe"])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "group": rng.choice([32, 64, 128]),
            "symmetric": rng.random() < 0.5}
    if op == "moe":
        E = _spread(rng, 4, 128)
        T = _spread(rng, 1, 64)
        H = _spread(rng, 256, 8192)
        F = _spread(rng, 256, min(11008, max(256, LARGEST_EXPERTS // (3 * E * H))))
        while 3 * E * H * F > LARGEST_EXPERTS:
            H = max(256, H // 2)
        case.update(T=T, E=E, k=rng.randint(1, min(8, E)), H=H, F=F, renormalize=rng.random() < 0.5,
                    activation=rng.choice(["silu", "gelu"]))
        return case
    M = _spread(rng, 256, 49152)
    K = _spread(rng, 256, min(49152, LARGEST_WEIGHT // M))
    if op == "encode":
        K = min(K, max(256, 36864 * 12288 // M))
    else:
        N = _spread(rng, 1, 256)
        # no more products than the largest listed case
        N = min(N, max(1, 9216 * 36864 * 256 // (M * K)))
        case.update(N=N)
    case.update(M=M, K=K)
    return case


def _groups(K, group):
    return -(-K // group)


def _weight(gen, shape, group, dtype, symmetric, device):
    """Codes with a bell-shaped histogram, scales of a few percent over their range, zero points near the middle."""
    codes = torch.randint(0, 8, shape, dtype=torch.uint8, device=device, generator=gen)
    codes += torch.randint(0, 9, shape, dtype=torch.uint8, device=device, generator=gen)
    per_group = (*shape[:-1], _groups(shape[-1], group))
    scales = torch.rand(per_group, device=device, generator=gen).mul_(0.004).add_(0.004).to(dtype)
    zeros = None if symmetric else torch.randint(5, 11, per_group, dtype=torch.uint8, device=device, generator=gen)
    return codes, scales, zeros


def _inputs(case, seed):
    """The inputs of a case as dense tensors and (codes, scales, zeros) triples, from the seed alone."""
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(int(seed))
    dtype, group, symmetric = TYPES[case["dtype"]], case["group"], case["symmetric"]
    if case["op"] == "encode":
        # trained weights: normal, with rows of different size
        rows = torch.rand((case["M"], 1), device=device, generator=gen).mul_(0.03).add_(0.01)
        W = torch.randn((case["M"], case["K"]), device=device, generator=gen).mul_(rows).to(dtype)
        return {"W": W}
    if case["op"] == "matmul":
        A = _weight(gen, (case["M"], case["K"]), group, dtype, symmetric, device)
        B = torch.randn((case["N"], case["K"]), device=device, generator=gen).to(dtype)
        return {"A": A, "B": B}
    E, H, F = case["E"], case["H"], case["F"]
    return {"X": torch.randn((case["T"], H), device=device, generator=gen).to(dtype),
            "router": torch.randn((E, H), device=device, generator=gen).mul_(1.5 / H ** 0.5).to(dtype),
            "gate": _weight(gen, (E, F, H), group, dtype, symmetric, device),
            "up": _weight(gen, (E, F, H), group, dtype, symmetric, device),
            "down": _weight(gen, (E, H, F), group, dtype, symmetric, device)}


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own:  # a program that serves a model keeps the weights in the package's layout
        import unstructured_sparse_skinny_b200 as fs
        for name in ("A", "gate", "up", "down"):
            if name in state:
                codes, scales, zeros = state[name]
                state[name] = fs.w4_pack(codes, scales, zeros, group=case["group"])
    return state


# ---------------------------------------------------------------- the plain form


def _dense(weight, group):
    """s * (q - z) in fp32."""
    codes, scales, zeros = weight
    K = codes.shape[-1]
    G = scales.shape[-1]
    q = codes.float()
    if K < G * group:
        q = torch.nn.functional.pad(q, (0, G * group - K))
    q = q.view(*codes.shape[:-1], G, group)
    q -= 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    q *= scales.float().unsqueeze(-1)
    return q.view(*codes.shape[:-1], G * group)[..., :K]


def _plain_encode(W, group, symmetric):
    M, K = W.shape
    G = _groups(K, group)
    w = W.float()
    if K < G * group:
        w = torch.nn.functional.pad(w, (0, G * group - K))
    w = w.view(M, G, group)
    if symmetric:
        s = (w.abs().amax(-1) / torch.tensor(7.0, device=W.device)).to(W.dtype)
    else:
        low, high = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
        s = ((high - low) / torch.tensor(15.0, device=W.device)).to(W.dtype)
    sf = s.float()
    div = torch.where(sf == 0, torch.ones_like(sf), sf)
    z = torch.full_like(sf, 8.0) if symmetric else (-low / div).round().clamp(0, 15)
    q = ((w / div.unsqueeze(-1)).round() + z.unsqueeze(-1)).clamp(0, 15)
    q -= z.unsqueeze(-1)
    q *= sf.unsqueeze(-1)
    return q.view(M, G * group)[:, :K].to(W.dtype)


def _act(name, g):
    return g * torch.sigmoid(g) if name == "silu" else 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5))


def _plain_moe(state):
    case, X = state["case"], state["X"]
    T, E, k, group = case["T"], case["E"], case["k"], case["group"]
    logits = X.double() @ state["router"].double().t()
    order = logits.sort(dim=1, descending=True, stable=True)
    ids, best = order.indices[:, :k], order.values[:, :k]
    top = order.values[:, :1]
    e = (best - top).float().exp()
    weights = e / (e.sum(1, keepdim=True) if case["renormalize"] else (logits - top).float().exp().sum(1, keepdim=True))
    x = X.float()
    if T * k <= E:  # few tokens: the chosen experts only
        pick = ids.reshape(-1)
        gate, up, down = (_dense(tuple(None if t is None else t[pick] for t in state[n]), group)
                          for n in ("gate", "up", "down"))
        xs = x.repeat_interleave(k, 0).unsqueeze(-1)
        h = _act(case["activation"], gate @ xs) * (up @ xs)
        out = ((down @ h).view(T, k, -1) * weights.unsqueeze(-1)).sum(1)
    else:  # most experts run: all of them for all tokens, those not chosen with weight zero
        h = _act(case["activation"], x @ _dense(state["gate"], group).transpose(1, 2))
        h *= x @ _dense(state["up"], group).transpose(1, 2)
        share = torch.zeros((T, E), device=X.device).scatter_(1, ids, weights)
        out = ((h @ _dense(state["down"], group).transpose(1, 2)) * share.t().unsqueeze(-1)).sum(0)
    return {"out": out.to(X.dtype), "ids": ids.to(torch.int32), "weights": weights}


def run(state):
    case = state["case"]
    if own:
        import unstructured_sparse_skinny_b200 as fs
        if case["op"] == "encode":
            return fs.w4_decode(fs.w4_encode(state["W"], group=case["group"], symmetric=case["symmetric"]))
        if case["op"] == "matmul":
            return fs.w4_matmul(state["A"], state["B"])
        out, ids, weights = fs.moe_w4(state["X"], state["router"], state["gate"], state["up"], state["down"], case["k"],
                                      renormalize=case["renormalize"], activation=case["activation"])
        return {"out": out, "ids": ids, "weights": weights}
    if case["op"] == "encode":
        return _plain_encode(state["W"], case["group"], case["symmetric"])
    if case["op"] == "matmul":
        return (state["B"].float() @ _dense(state["A"], case["group"]).t()).to(state["B"].dtype)
    return _plain_moe(state)


# ---------------------------------------------------------------- work and 64-bit values


def _weight_bytes(M, K, group, symmetric):
    """Half a byte a value, two bytes a scale, one byte a zero point."""
    return M * K / 2 + M * _groups(K, group) * (2 if symmetric else 3)


def work(case):
    group, symmetric = case["group"], case["symmetric"]
    if case["op"] == "encode":
        M, K = case["M"], case["K"]
        # the dense weight in and out, the encoded one written and read
        return {"bytes": 4 * M * K + 2 * _weight_bytes(M, K, group, symmetric), "flops": 6 * M * K}
    if case["op"] == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": _weight_bytes(M, K, group, symmetric) + 2 * N * (K + M), "flops": 2 * M * K * N}
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    running = E * (1 - (1 - k / E) ** T)  # experts that some token chose, for even routing
    bytes_ = 2 * E * H + running * (2 * _weight_bytes(F, H, group, symmetric) + _weight_bytes(H, F, group, symmetric))
    return {"bytes": bytes_ + 4 * T * H + 8 * T * k, "flops": 2 * T * E * H + 6 * T * k * H * F}


def _exact_weight(weight, index, group):
    """One matrix in fp64, its groups' scales spelled out for every column."""
    codes, scales, zeros = (t if t is None or index is None else t[index] for t in weight)
    of = torch.arange(codes.shape[1], device=codes.device) // group
    z = 8.0 if zeros is None else zeros.double()[:, of]
    return (codes.double() - z) * scales.double()[:, of]


def exact(case, seed):
    data, group = _inputs(case, seed), case["group"]
    if case["op"] == "encode":
        W = data["W"]
        out = torch.empty_like(W, dtype=torch.float64)
        for k0 in range(0, W.shape[1], group):  # group by group
            w = W[:, k0:k0 + group].double()
            if case["symmetric"]:
                s = (w.abs().max(1, keepdim=True).values / 7).to(W.dtype).double()
                zero = torch.full_like(s, 8)
            else:
                low = torch.minimum(w.min(1, keepdim=True).values, torch.zeros_like(w[:, :1]))
                high = torch.maximum(w.max(1, keepdim=True).values, torch.zeros_like(w[:, :1]))
                s = ((high - low) / 15).to(W.dtype).double()
                zero = torch.where(s > 0, torch.round(-low / s.clamp(min=1e-300)), torch.zeros_like(s)).clamp(0, 15)
            q = torch.where(s > 0, torch.round(w / s.clamp(min=1e-300)) + zero, zero).clamp(0, 15)
            out[:, k0:k0 + group] = s * (q - zero)
        return out
    if case["op"] == "matmul":
        rows = max(1, (1 << 28) // case["K"])
        B = data["B"].double()
        parts = []
        for m0 in range(0, case["M"], rows):
            part = tuple(None if t is None else t[m0:m0 + rows] for t in data["A"])
            parts.append(B @ _exact_weight(part, None, group).t())
        return torch.cat(parts, 1)
    X, k = data["X"].double(), case["k"]
    p = torch.softmax(X @ data["router"].double().t(), 1)
    weights, ids = p.sort(dim=1, descending=True, stable=True)
    weights, ids = weights[:, :k], ids[:, :k]
    if case["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    out = torch.zeros_like(X)
    for e in range(case["E"]):
        token, place = (ids == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        g = X[token] @ _exact_weight(data["gate"], e, group).t()
        u = X[token] @ _exact_weight(data["up"], e, group).t()
        g = torch.nn.functional.silu(g) if case["activation"] == "silu" else torch.nn.functional.gelu(g)
        out.index_add_(0, token, (g * u) @ _exact_weight(data["down"], e, group).t() * weights[token, place].unsqueeze(1))
    return {"out": out, "ids": None, "weights": weights}

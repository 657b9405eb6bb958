"""Cases of the 8-bit integer operators: what is computed, on which inputs, and how much work it is.

Four operators that run one after another around a frozen, masked linear:

  linear    Y = (Xq . (Wq (.) Mask)^T) * x_scale[m] * w_scale[n], 8-bit integer codes with one scale per
            token and one per output channel, over a weight whose tiles are dense or 2:4 sparse
  rmsnorm   h = x + residual; the codes and scales of h / rms(h) * gamma
  silu_mul  the codes and scales of silu(gate) * up
  quantize  the codes and scales of x

Codes: scale[m] = max(max_k |y[m, k]| / 127, 2^-126), code = round(y / scale), ties to even. Outputs held in
8 bits are returned as the values they stand for, in bf16.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls that a user
of the package makes. Sizes are those of the Llama-shaped linears that the tests and the benchmark use.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
SMALLEST_SCALE = 2.0 ** -126


def listed():
    return [
        # one token through an attention projection: the smallest call, where latency counts
        {"name": "linear_m1", "op": "linear", "M": 1, "N": 4096, "K": 4096, "rows": 128, "cols": 128, "sparse": 0.7,
         "out": "bf16", "pad": 0},
        # a decode batch through the up projection
        {"name": "linear_m16", "op": "linear", "M": 16, "N": 11008, "K": 4096, "rows": 128, "cols": 128, "sparse": 0.7,
         "out": "bf16", "pad": 0},
        # a short ragged prompt through the down projection: small mask tiles, input rows with a pitch
        {"name": "linear_m100", "op": "linear", "M": 100, "N": 4096, "K": 11008, "rows": 64, "cols": 64, "sparse": 0.7,
         "out": "fp16", "pad": 64},
        # prefill of one sequence through the gate projection
        {"name": "linear_m2048", "op": "linear", "M": 2048, "N": 11008, "K": 4096, "rows": 128, "cols": 128,
         "sparse": 0.9, "out": "bf16", "pad": 0},
        # prefill of a batch of sequences, the largest call
        {"name": "linear_m8192", "op": "linear", "M": 8192, "N": 13824, "K": 5120, "rows": 128, "cols": 64,
         "sparse": 0.9, "out": "bf16", "pad": 0},
        # the norm ahead of the attention in a decode step
        {"name": "rmsnorm_m1", "op": "rmsnorm", "M": 1, "K": 4096, "type": "bf16", "residual": True, "pad": 0},
        # the same over a ragged prefill, no residual yet (the first layer)
        {"name": "rmsnorm_m777", "op": "rmsnorm", "M": 777, "K": 2048, "type": "fp16", "residual": False, "pad": 0},
        # and over a batch of sequences
        {"name": "rmsnorm_m8192", "op": "rmsnorm", "M": 8192, "K": 5120, "type": "bf16", "residual": True, "pad": 0},
        # the activation of a decode batch, gate and up apart
        {"name": "silu_mul_m16", "op": "silu_mul", "M": 16, "K": 11008, "type": "bf16", "joined": False},
        # the activation of a prefill, gate and up side by side in one matrix
        {"name": "silu_mul_m4096", "op": "silu_mul", "M": 4096, "K": 8192, "type": "bf16", "joined": True},
        # the attention's output ahead of its projection: a decode batch, and a batch of sequences
        {"name": "quantize_m16", "op": "quantize", "M": 16, "K": 4096, "type": "fp16", "pad": 0},
        {"name": "quantize_m8192", "op": "quantize", "M": 8192, "K": 5120, "type": "bf16", "pad": 64},
    ]


def spread(rng, low, high):
    """A whole number in [low, high], even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rmsnorm", "silu_mul", "quantize"])
    if op == "linear":
        rows, cols = rng.choice([(128, 128), (128, 64), (64, 128), (64, 64)])
        n, k = 128 * spread(rng, 1, 108), cols * spread(rng, 1, 13824 // cols)
        m = spread(rng, 1, min(8192, 8192 * 13824 * 5120 // (n * k)))
        return {"op": op, "M": m, "N": n, "K": k, "rows": rows, "cols": cols, "sparse": rng.choice([0.0, 0.5, 0.7, 0.9, 1.0]),
                "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "pad": rng.choice([0, 0, 16, 64])}
    case = {"op": op, "M": spread(rng, 1, 8192), "K": spread(rng, 64, 13824 if op == "silu_mul" else 8192),
            "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    case["M"] = min(case["M"], 8192 * 5120 // case["K"])
    if op == "rmsnorm":
        case["residual"] = rng.random() < 0.7
    if op == "silu_mul":
        case["joined"] = rng.random() < 0.5
    else:
        case["pad"] = rng.choice([0, 0, 1, 8, 64])
    return case


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def rows_of(values, pad):
    """`values` as the first columns of a wider matrix: rows with a pitch of K + pad."""
    if not pad:
        return values
    wide = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device=values.device)
    wide[:, :values.shape[1]] = values
    return wide[:, :values.shape[1]]


def activations(g, m, k):
    """Token rows of unequal size, with a few channels that stand out, as the layers' hidden states have them."""
    x = normal(g, m, k) * torch.exp(0.5 * normal(g, m, 1))
    loud = torch.rand(k, generator=g, device="cuda") < 0.004
    return x * torch.where(loud, 12.0, 1.0)


def prepare_linear(case, seed):
    g = generator(seed)
    m, n, k, rows, cols = case["M"], case["N"], case["K"], case["rows"], case["cols"]
    w = normal(g, n, k) * 0.02
    tiles = (n // rows) * (k // cols)
    flags = torch.zeros(tiles, dtype=torch.uint8, device="cuda")
    flags[torch.randperm(tiles, generator=g, device="cuda")[:round(case["sparse"] * tiles)]] = 1
    flags = flags.view(n // rows, k // cols)
    # a 2:4 tile keeps the two largest of every four weights along k
    kept = torch.zeros(n * k // 4, 4, dtype=torch.bool, device="cuda")
    kept.scatter_(1, w.abs().view(-1, 4).topk(2, dim=1).indices, True)
    kept = kept.view(n, k) | ~flags.bool().repeat_interleave(rows, 0).repeat_interleave(cols, 1)
    w = w * kept
    w_scale = (w.abs().amax(1) / 127).clamp_min(SMALLEST_SCALE)
    codes = torch.round(w / w_scale[:, None]).to(torch.int8)
    x = activations(g, m, k)
    x_scale = (x.abs().amax(1) / 127).clamp_min(SMALLEST_SCALE)
    state = {"case": case, "x": rows_of(torch.round(x / x_scale[:, None]).to(torch.int8), case["pad"]), "x_scale": x_scale,
             "w": codes, "w_scale": w_scale}
    if own:
        import hybrid_sparse_gemm_b200 as hsg
        weights = torch.tensor([128, 64, 32, 16, 8, 4, 2, 1], dtype=torch.uint8, device="cuda")
        bits = (kept.view(-1, 8) * weights).sum(1, dtype=torch.uint8)
        state["linear"] = hsg.PackedLinearQ8.pack(codes, bits, flags.cpu(), rows, cols, w_scale=w_scale)
        state["out"] = torch.empty(m, n, dtype=TYPES[case["out"]], device="cuda")
    return state


def prepare(case, seed):
    if case["op"] == "linear":
        return prepare_linear(case, seed)
    g = generator(seed)
    m, k, t = case["M"], case["K"], TYPES[case["type"]]
    state = {"case": case}
    if case["op"] == "silu_mul":
        gate, up = (2 * normal(g, m, k)).to(t), activations(g, m, k).to(t)
        if case["joined"]:
            both = torch.cat([gate, up], 1)
            gate, up = both[:, :k], both[:, k:]
        state.update(gate=gate, up=up)
    else:
        state["x"] = rows_of(activations(g, m, k).to(t), case["pad"])
    if case["op"] == "rmsnorm":
        state["gamma"] = (1 + 0.2 * normal(g, k)).to(t)
        state["residual"] = rows_of((3 * activations(g, m, k)).to(t), case["pad"]) if case["residual"] else None
    state["values"] = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    if own:
        state["codes"] = torch.empty(m, k, dtype=torch.int8, device="cuda")
        state["scale"] = torch.empty(m, dtype=torch.float32, device="cuda")
        state["stream"] = torch.empty(m, k, dtype=t, device="cuda")
    return state


def coded(y, values):
    """The codes and scales of the rows of y, as (values that the codes stand for, scales)."""
    scale = (y.abs().amax(1) / 127).clamp_min(SMALLEST_SCALE)
    torch.mul(torch.round(y / scale[:, None]).to(torch.int8), scale[:, None], out=values)
    return {"values": values, "scale": scale}


def run_own(s):
    import hybrid_sparse_gemm_b200 as hsg
    op = s["case"]["op"]
    if op == "linear":
        return {"y": s["linear"](s["x"], s["x_scale"], out=s["out"])}
    out = {"scale": s["scale"]}
    if op == "quantize":
        hsg.patch_quantize_q8(s["x"], s["codes"], s["scale"])
    elif op == "silu_mul":
        hsg.patch_silu_mul_q8(s["gate"], s["up"], s["codes"], s["scale"])
    elif s["residual"] is None:
        hsg.patch_rmsnorm_q8(s["x"], s["gamma"], EPS, s["codes"], s["scale"])
    else:
        hsg.patch_rmsnorm_q8(s["x"], s["gamma"], EPS, s["codes"], s["scale"], residual=s["residual"],
                             residual_out=s["stream"])
        out["residual"] = s["stream"]
    hsg.patch_dequantize_q8(s["codes"], s["scale"], s["values"])
    out["values"] = s["values"]
    return out


def run(s):
    if own:
        return run_own(s)
    op = s["case"]["op"]
    if op == "linear":
        y = s["x"].float() @ s["w"].float().t()
        return {"y": (y * s["x_scale"][:, None] * s["w_scale"]).to(TYPES[s["case"]["out"]])}
    if op == "quantize":
        return coded(s["x"].float(), s["values"])
    if op == "silu_mul":
        gate = s["gate"].float()
        return coded(gate / (1 + torch.exp(-gate)) * s["up"].float(), s["values"])
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(s["x"].dtype)
        stream, h = h, h.float()
    out = coded(h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["gamma"].float(), s["values"])
    if s["residual"] is not None:
        out["residual"] = stream
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        total = torch.mm(s["x"].to(torch.float64), s["w"].to(torch.float64).t())  # whole numbers below 2^53
        total *= s["x_scale"].to(torch.float64).unsqueeze(1)
        total *= s["w_scale"].to(torch.float64).unsqueeze(0)
        return {"y": total}
    answer = {}
    if case["op"] == "quantize":
        y = s["x"].to(torch.float64)
    elif case["op"] == "silu_mul":
        y = s["gate"].to(torch.float64) * torch.sigmoid(s["gate"].to(torch.float64)) * s["up"].to(torch.float64)
    else:
        h = s["x"].to(torch.float64)
        if case["residual"]:
            h = h + s["residual"].to(torch.float64)
            answer["residual"] = h
            h = h.to(s["x"].dtype).to(torch.float64)  # the norm is that of the stored sum
        y = h * s["gamma"].to(torch.float64) / torch.sqrt((h * h).sum(1) / case["K"] + EPS).unsqueeze(1)
    scale = torch.clamp(y.abs().max(1).values / 127.0, min=SMALLEST_SCALE)
    answer["scale"] = scale
    answer["values"] = torch.round(y / scale.unsqueeze(1)) * scale.unsqueeze(1)
    return answer


def work(case):
    m, k = case["M"], case["K"]
    if case["op"] == "linear":
        n = case["N"]
        tiles = (n // case["rows"]) * (k // case["cols"])
        sparse = round(case["sparse"] * tiles) / tiles  # of the weights, in 2:4 tiles: half a byte and a bit each
        return {"bytes": m * k + 4 * m + n * k * (1 - sparse + 0.625 * sparse) + 4 * n + m * n * BYTES[case["out"]],
                "flops": 2.0 * m * n * k * (1 - 0.5 * sparse)}
    size = BYTES[case["type"]]
    written = m * k + 4 * m
    if case["op"] == "quantize":
        return {"bytes": m * k * size + written, "flops": 3.0 * m * k}
    if case["op"] == "silu_mul":
        return {"bytes": 2 * m * k * size + written, "flops": 8.0 * m * k}
    moved = (3 if case["residual"] else 1) * m * k + k
    return {"bytes": moved * size + written, "flops": 7.0 * m * k}

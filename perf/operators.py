"""The gated feed-forward and adapter operators: what they are measured on.

Four operators around a decoder's feed-forward block whose weights are ternary:

  glu            h = act(x Wg^T) * (x Wu^T) on packed ternary gate and up weights (serving)
  lora           y = x W^T + s_a (x A_a^T) B_a^T: a packed ternary projection shared by all rows
                 beside the low-rank adapter a that each row's request names (serving)
  glu_forward    the gated block on the bf16 weights that quantization-aware training multiplies by
  glu_backward   its gradients with respect to x and both weights

Sizes are those of the two feed-forward blocks the repository is configured
for, hidden 1024 / intermediate 3584 and hidden 4096 / intermediate 14336, and
odd ones between them.
"""
import math

import torch

own = False

# Bytes a group: five base-3 digits a byte, each group padded to whole bytes.
_GROUP_BYTES = {64: 13, 128: 26}


def listed():
    return [
        # One token through the smaller block's gate and up: latency alone.
        {"name": "glu token", "op": "glu", "M": 1, "N": 3584, "K": 1024, "G": 128, "act": "silu"},
        # A few sequences decoded together through the larger block, finer groups.
        {"name": "glu decode 7", "op": "glu", "M": 7, "N": 14336, "K": 4096, "G": 64, "act": "silu"},
        # A short ragged prompt, the other activation.
        {"name": "glu prompt 333", "op": "glu", "M": 333, "N": 3584, "K": 1024, "G": 128, "act": "gelu"},
        # A long prompt through the larger block: matrix work.
        {"name": "glu prompt 2048", "op": "glu", "M": 2048, "N": 14336, "K": 4096, "G": 128, "act": "silu"},
        # One token of one request's adapter on the smaller block's down projection.
        {"name": "lora token", "op": "lora", "M": 1, "N": 1024, "K": 3584, "G": 128, "R": 8,
         "adapters": 4, "rows": "each"},
        # A decode batch in which every request has an adapter of its own (some none).
        {"name": "lora decode 32", "op": "lora", "M": 32, "N": 4096, "K": 14336, "G": 128, "R": 16,
         "adapters": 32, "rows": "each"},
        # Prompts of several requests laid end to end, higher rank.
        {"name": "lora prompts 1900", "op": "lora", "M": 1900, "N": 4096, "K": 14336, "G": 128,
         "R": 64, "adapters": 6, "rows": "runs"},
        # A small training batch with sizes that fill no tile.
        {"name": "forward 75", "op": "glu_forward", "M": 75, "N": 700, "K": 512, "act": "gelu"},
        # The smaller block's training batch: 8 sequences of 512.
        {"name": "forward 4096", "op": "glu_forward", "M": 4096, "N": 3584, "K": 1024, "act": "silu"},
        # The gradients of a short batch: the three products have little to share the chip with.
        {"name": "backward 129", "op": "glu_backward", "M": 129, "N": 3584, "K": 1024, "act": "gelu"},
        # The smaller block's training batch, backwards.
        {"name": "backward 4096", "op": "glu_backward", "M": 4096, "N": 3584, "K": 1024, "act": "silu"},
        # The larger block: the most work of all.
        {"name": "backward 2048 wide", "op": "glu_backward", "M": 2048, "N": 14336, "K": 4096,
         "act": "silu"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["glu", "glu", "lora", "lora", "glu_forward", "glu_backward"])
    G = rng.choice([64, 128])
    # an odd number of groups a row, or one of the two blocks' widths
    if rng.random() < 0.6:
        top = 14336 if op == "lora" else 4096
        K = G * (2 * (spread(256, top) // (2 * G)) + 1)
        N = spread(256, 4096 if op == "lora" else 14336) | 1 if rng.random() < 0.5 else \
            16 * (2 * (spread(256, 14336 if op != "lora" else 4096) // 32) + 1)
    else:
        N, K = rng.choice([(3584, 1024), (14336, 4096)])
        if op == "lora":
            N, K = K, N
    limit = {"glu": 2048 * 14336 * 4096, "lora": 1900 * 4096 * 14336,
             "glu_forward": 4096 * 3584 * 1024, "glu_backward": 2048 * 14336 * 4096}[op]
    if op in ("glu", "lora") and rng.random() < 0.4:
        M = spread(1, 64)
    else:
        M = spread(1, 4096)
    M = max(1, min(M, limit // (N * K)))
    case = {"op": op, "M": M, "N": N, "K": K}
    if op in ("glu", "lora"):
        case["G"] = G
    if op == "lora":
        case["R"] = rng.choice([8, 16, 24, 32, 64])
        case["rows"] = rng.choice(["each", "runs"])
        case["adapters"] = min(rng.choice([1, 3, 8, 20, 32]), max(1, M // 8) if case["rows"] == "runs" else 32)
    else:
        case["act"] = rng.choice(["silu", "gelu"])
    if op in ("glu_forward", "glu_backward") and K * N * M > limit:
        case["N"] = max(16, limit // (K * M))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _codes(g, shape):
    """Ternary codes as an absmean rule leaves them on normal weights: about
    three in ten are zero."""
    r = torch.rand(shape, generator=g, device="cuda")
    return (r > 0.65).to(torch.uint8) + (r > 0.35).to(torch.uint8)      # digit = code + 1


def _scales(g, shape):
    """Group scales as such weights have them: near 0.016, a tenth apart."""
    return (0.016 * torch.exp(0.1 * torch.randn(shape, generator=g, device="cuda"))).to(torch.float16)


def _packed(g, N, K, G):
    nG, B = K // G, _GROUP_BYTES[G]
    d = _codes(g, (N, nG, 5 * B))
    d[:, :, G:] = 1                                                      # padding: code 0
    d = d.view(N, nG, B, 5)
    p = d[..., 0] + 3 * d[..., 1] + 9 * d[..., 2] + 27 * d[..., 3] + 81 * d[..., 4]
    return p.reshape(N, nG * B).contiguous(), _scales(g, (N, nG))


def _ternary_bf16(g, N, K):
    """The bf16 weights quantization-aware training multiplies by: codes times
    the scale of each 64."""
    c = _codes(g, (N, K)).to(torch.float32) - 1.0
    s = _scales(g, (N, K // 64 if K % 64 == 0 else 1)).to(torch.float32)
    return (c.view(N, s.shape[1], -1) * s[..., None]).view(N, K).to(torch.bfloat16)


def _active(M):
    """Rows with an adapter where every request has its own: one in eight has none."""
    return M - M // 8


def _ids(g, case):
    M, n = case["M"], case["adapters"]
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    row = torch.arange(M, device="cuda")
    if case["rows"] == "each":
        return torch.where(row % 8 == 7, torch.full_like(row, -1, dtype=torch.int32),
                           order[(row - row // 8) % n]).to(torch.int32)
    # runs: the prompts of n requests end to end, of uneven lengths, none empty
    w = torch.rand(n, generator=g, device="cuda") + 0.2
    ends = torch.cumsum(w, 0) / w.sum() * (M - n)
    ends = ends.floor().to(torch.int64) + torch.arange(1, n + 1, device="cuda")
    ends[-1] = M
    return order[torch.searchsorted(ends, row, right=True)].contiguous()


def _inputs(case, seed):
    g = _gen(seed)
    M, N, K = case["M"], case["N"], case["K"]
    s = {"x": _normal(g, (M, K))}
    if case["op"] == "glu":
        s["gate"] = _packed(g, N, K, case["G"])
        s["up"] = _packed(g, N, K, case["G"])
    elif case["op"] == "lora":
        R, n = case["R"], case["adapters"]
        s["w"] = _packed(g, N, K, case["G"])
        s["ids"] = _ids(g, case)
        s["a"] = _normal(g, (n, R, K), K ** -0.5)
        s["b"] = _normal(g, (n, N, R), 0.2)
        s["scaling"] = 0.5 + torch.rand(n, generator=g, device="cuda")
    else:
        s["wg"] = _ternary_bf16(g, N, K)
        s["wu"] = _ternary_bf16(g, N, K)
        if case["op"] == "glu_backward":
            s["dh"] = _normal(g, (M, N))
            s["g"] = (s["x"].float() @ s["wg"].float().t()).to(torch.bfloat16)
            s["u"] = (s["x"].float() @ s["wu"].float().t()).to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import ternary_weight_only_amd as tq
        s["tq"] = tq
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    tq, c = s["tq"], s["case"]
    if c["op"] == "glu":
        return tq.glu(s["x"], s["gate"], s["up"], c["N"], c["K"], c["G"], act=c["act"])
    if c["op"] == "lora":
        return tq.lora_matmul(s["x"], s["w"][0], s["w"][1], s["ids"], s["a"], s["b"], s["scaling"],
                              c["N"], c["K"], c["G"])
    if c["op"] == "glu_forward":
        return tq.glu_forward(s["x"], s["wg"], s["wu"], act=c["act"])        # h, g, u
    return tq.glu_backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], act=c["act"])


def _unpack(packed, scales, N, K, G):
    nG, B = K // G, _GROUP_BYTES[G]
    p = packed.view(N, nG, B, 1).to(torch.int16)
    powers = torch.tensor([1, 3, 9, 27, 81], dtype=torch.int16, device=packed.device)
    digit = torch.remainder(torch.div(p, powers, rounding_mode="floor"), 3)
    code = digit.view(N, nG, 5 * B)[:, :, :G].to(torch.float32) - 1.0
    return (code * scales.view(N, nG, 1).to(torch.float32)).view(N, K)


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return sg * (1.0 + g * (1.0 - sg))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    x = s["x"].to(torch.float32)
    if c["op"] == "glu":
        g = x @ _unpack(*s["gate"], N, K, c["G"]).t()
        u = x @ _unpack(*s["up"], N, K, c["G"]).t()
        return (_act(g, c["act"]) * u).to(torch.bfloat16)
    if c["op"] == "lora":
        y = x @ _unpack(*s["w"], N, K, c["G"]).t()
        for a in range(c["adapters"]):
            add = s["scaling"][a] * ((x @ s["a"][a].to(torch.float32).t()) @ s["b"][a].to(torch.float32).t())
            y = torch.where((s["ids"] == a)[:, None], y + add, y)
        return y
    wg, wu = s["wg"].to(torch.float32), s["wu"].to(torch.float32)
    if c["op"] == "glu_forward":
        g, u = x @ wg.t(), x @ wu.t()
        h = _act(g, c["act"]) * u
        return h.to(torch.bfloat16), g.to(torch.bfloat16), u.to(torch.bfloat16)
    g, u, dh = s["g"].to(torch.float32), s["u"].to(torch.float32), s["dh"].to(torch.float32)
    dg = dh * u * _act_slope(g, c["act"])
    du = dh * _act(g, c["act"])
    dx = dg @ wg + du @ wu
    return (dx.to(torch.bfloat16), (dg.t() @ x).to(torch.bfloat16), (du.t() @ x).to(torch.bfloat16))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] in ("glu", "lora"):
        weights = N * (K // case["G"]) * (_GROUP_BYTES[case["G"]] + 2)
    if case["op"] == "glu":
        return {"bytes": 2 * weights + 2 * M * K + 2 * M * N, "flops": 4 * M * N * K}
    if case["op"] == "lora":
        rows = _active(M) if case["rows"] == "each" else M
        used = min(case["adapters"], rows)
        return {"bytes": weights + 2 * M * K + 4 * M * N + 4 * M + used * (2 * case["R"] * (K + N) + 4),
                "flops": 2 * M * N * K + 2 * rows * case["R"] * (N + K)}
    if case["op"] == "glu_forward":
        return {"bytes": 2 * M * K + 4 * N * K + 6 * M * N, "flops": 4 * M * N * K}
    return {"bytes": 6 * M * N + 4 * M * K + 8 * N * K, "flops": 8 * M * N * K}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _weights64(packed, scales, N, K, G):
    """Every byte value's five digits looked up, times the group's scale."""
    table = torch.tensor([[v // 3 ** i % 3 - 1 for i in range(5)] for v in range(243)],
                         dtype=torch.int8, device=packed.device)
    rows = table[packed.to(torch.int32)].view(N * (K // G), -1)[:, :G]
    return (rows.to(torch.float64) * scales.to(torch.float64).view(-1, 1)).view(N, K)


def _gates64(g, act):
    """The activation and its derivative."""
    if act == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig + g * sig * (1 - sig)
    inner = (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    half = torch.sigmoid(2 * inner)                    # (1 + tanh(z)) / 2 = sigmoid(2 z)
    slope = (2 / math.pi) ** 0.5 * (1 + 0.134145 * g ** 2)
    return g * half, half + 2 * g * half * (1 - half) * slope


def exact(case, seed):
    s = _inputs(case, seed)
    N, K = case["N"], case["K"]
    x = s["x"].double()
    if case["op"] == "glu":
        g = torch.mm(x, _weights64(*s["gate"], N, K, case["G"]).t())
        u = torch.mm(x, _weights64(*s["up"], N, K, case["G"]).t())
        return _gates64(g, case["act"])[0] * u
    if case["op"] == "lora":
        y = torch.mm(x, _weights64(*s["w"], N, K, case["G"]).t())
        for a in sorted(set(s["ids"].tolist()) - {-1}):
            at = (s["ids"] == a).nonzero()[:, 0]
            low = torch.mm(x[at], s["a"][a].double().t()) * s["scaling"][a].double()
            y[at] += torch.mm(low, s["b"][a].double().t())
        return y
    wg, wu = s["wg"].double(), s["wu"].double()
    if case["op"] == "glu_forward":
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        return _gates64(g, case["act"])[0] * u, g, u
    value, slope = _gates64(s["g"].double(), case["act"])
    dg = s["dh"].double() * s["u"].double() * slope
    du = s["dh"].double() * value
    return (torch.mm(dg, wg) + torch.mm(du, wu), torch.mm(dg.t().contiguous(), x),
            torch.mm(du.t().contiguous(), x))

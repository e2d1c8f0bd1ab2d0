"""Operators of a ternary model whose activations are held in 8 bits: what they are measured on.

  norm       the root-mean-square norm in front of a projection: the residual's addition, the norm and
             the rounding of each row to 8 bits with a scale, as the values those stand for (what
             quantization-aware training multiplies by); forward and backward
  norm_i8    the same for serving, followed by the projection that reads its 8-bit rows
  gemm       rows in 8 bits times packed ternary weights, with bias, activation and residual in the
             epilogue (serving)
  experts    the same product grouped by expert: rows sorted by expert, each segment of any length
             times its expert's packed weights (serving)

Sizes are those of the two feed-forward blocks the repository is configured
for, hidden 1024 / intermediate 3584 and hidden 4096 / intermediate 14336, and
odd ones between them.
"""
import math

import torch

own = False

EPS = 1e-6

# Bytes a group: five base-3 digits a byte, each group padded to whole bytes.
_GROUP_BYTES = {64: 13, 128: 26}


def listed():
    return [
        # One token's hidden state: latency alone.
        {"name": "norm token", "op": "norm", "M": 1, "K": 1024, "stream": "bf16", "residual": True},
        # A training batch of the larger model: 8 sequences of 512.
        {"name": "norm forward 4096", "op": "norm", "M": 4096, "K": 4096, "stream": "bf16", "residual": True},
        # Backwards through the norm of a short batch whose residual stream is kept in fp32.
        {"name": "norm backward 333", "op": "norm_backward", "M": 333, "K": 3584, "stream": "fp32"},
        # The larger model's training batch, backwards.
        {"name": "norm backward 4096", "op": "norm_backward", "M": 4096, "K": 4096, "stream": "bf16"},
        # One token through a norm and the projection behind it: two launches' latency.
        {"name": "norm and product token", "op": "norm_i8", "M": 1, "N": 3584, "K": 1024, "G": 128,
         "act": "relu2", "bias": False, "residual": False, "out": "bf16"},
        # A few sequences decoded together through the larger up projection, finer groups.
        {"name": "product decode 7", "op": "gemm", "M": 7, "N": 14336, "K": 4096, "G": 64,
         "act": "silu", "bias": True, "residual": False, "out": "bf16"},
        # A short ragged prompt through the smaller down projection, back into the residual stream.
        {"name": "product prompt 333", "op": "gemm", "M": 333, "N": 1024, "K": 3584, "G": 128,
         "act": "none", "bias": True, "residual": True, "out": "fp32"},
        # A long prompt through the larger up projection: matrix work.
        {"name": "product prompt 2048", "op": "gemm", "M": 2048, "N": 14336, "K": 4096, "G": 128,
         "act": "relu2", "bias": False, "residual": False, "out": "bf16"},
        # Eight tokens decoded together, two experts of eight each.
        {"name": "experts decode 8", "op": "experts", "tokens": 8, "top": 2, "E": 8, "N": 3584, "K": 1024,
         "G": 128, "gather": True, "act": "relu2", "bias": False, "residual": False, "out": "bf16"},
        # The way back from the larger experts for 32 tokens, two of sixteen each: bound by the weights.
        {"name": "experts decode 32", "op": "experts", "tokens": 32, "top": 2, "E": 16, "N": 4096, "K": 14336,
         "G": 128, "gather": False, "act": "none", "bias": False, "residual": False, "out": "fp32"},
        # A prompt over many small experts: ragged segments, some shorter than a tile, some empty.
        {"name": "experts prompt 1000", "op": "experts", "tokens": 1000, "top": 2, "E": 32, "N": 3584, "K": 1024,
         "G": 64, "gather": True, "act": "gelu", "bias": True, "residual": False, "out": "bf16"},
        # A long prompt over the larger experts: the most work of all.
        {"name": "experts prompt 2048", "op": "experts", "tokens": 2048, "top": 2, "E": 8, "N": 14336, "K": 4096,
         "G": 128, "gather": True, "act": "relu2", "bias": False, "residual": False, "out": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_backward", "norm_i8", "gemm", "gemm", "experts", "experts", "experts"])
    if op in ("norm", "norm_backward"):
        K = rng.choice([1024, 3584, 4096, 14336]) if rng.random() < 0.4 else spread(64, 16384)
        case = {"op": op, "M": max(1, min(spread(1, 8192), 4096 * 4096 // K)), "K": K,
                "stream": rng.choice(["bf16", "bf16", "fp32"])}
        if op == "norm":
            case["residual"] = rng.random() < 0.7
        return case
    G = rng.choice([64, 128])
    # one of the two blocks' projections, or an odd number of groups a row
    if rng.random() < 0.4:
        N, K = rng.choice([(3584, 1024), (14336, 4096), (1024, 3584), (4096, 14336)])
    else:
        K = G * (2 * (spread(256, 14336) // (2 * G)) + 1)
        N = spread(256, 14336) | (1 if rng.random() < 0.5 else 0)
    case = {"op": op, "N": N, "K": K, "G": G, "act": rng.choice(["none", "silu", "gelu", "relu2"]),
            "bias": rng.random() < 0.5, "residual": rng.random() < 0.4, "out": rng.choice(["bf16", "bf16", "fp32"])}
    limit = 2048 * 14336 * 4096
    rows = spread(1, 64) if rng.random() < 0.4 else spread(1, 4096)
    rows = max(1, min(rows, limit // (N * K)))
    if op == "experts":
        case["E"] = min(rng.choice([2, 5, 8, 16, 32, 64]), max(2, 16 * 4096 * 14336 // (N * K)))
        case["top"] = min(rng.choice([1, 2, 2, 4]), case["E"])
        case["tokens"] = rows
        case["gather"] = rng.random() < 0.6
    else:
        case["M"] = rows
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(g, shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _packed(g, shape, K, G):
    """Ternary weights of a stack of matrices: codes -1, 0, 1 alike often, as an
    absmean rule leaves them nearly, and group scales near 0.016, a tenth apart."""
    nG, B = K // G, _GROUP_BYTES[G]
    p = torch.randint(0, 243, (*shape, nG, B), generator=g, device="cuda", dtype=torch.uint8)
    left = G - 5 * (B - 1)                               # codes of a group's last byte
    last = torch.randint(0, 3 ** left, (*shape, nG), generator=g, device="cuda", dtype=torch.int32)
    p[..., B - 1] = (last + sum(3 ** i for i in range(left, 5))).to(torch.uint8)   # then zero trits
    s = 0.016 * torch.exp(0.1 * torch.randn((*shape, nG), generator=g, device="cuda"))
    return p.view(*shape, nG * B), s.to(torch.float16)


def _rows_i8(g, M, K):
    """Normal activations as a norm leaves them: each row in 8 bits by its largest."""
    x = torch.randn((M, K), generator=g, device="cuda")
    top = x.abs().amax(1)
    return torch.round(x * (127.0 / top)[:, None]).to(torch.int8), top / 127.0


def _routes(g, case):
    """Experts of each token, `top` different ones, some experts liked more than
    others: (rows sorted by expert -> token, int32; segment ends, int32 [E + 1])."""
    t, n, E = case["tokens"], case["top"], case["E"]
    like = torch.rand((t, E), generator=g, device="cuda").log().neg().log().neg()
    like += 0.7 * torch.randn((1, E), generator=g, device="cuda")
    picked = like.topk(n, dim=1).indices.view(-1)
    order = torch.sort(picked, stable=True).indices
    ends = torch.cumsum((picked[:, None] == torch.arange(E, device="cuda")).sum(0), 0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ends]).to(torch.int32)
    return (order // n).to(torch.int32), offsets


def _inputs(case, seed):
    g = _gen(seed)
    op, K, s = case["op"], case["K"], {}
    if op in ("norm", "norm_i8"):
        M = case["M"]
        stream = _type(case.get("stream", "bf16"))
        # what the block before adds, and the stream it is added to: a few channels far above the others
        s["x"] = _normal(g, (M, K))
        if op == "norm_i8" or case["residual"]:
            wide = 1.0 + 20.0 * (torch.rand((1, K), generator=g, device="cuda") < 0.01).to(torch.float32)
            s["r"] = (3.0 * wide * torch.randn((M, K), generator=g, device="cuda")).to(stream)
        elif stream != torch.bfloat16:
            s["x"] = _normal(g, (M, K), 1.0, stream)
        s["w"] = (1.0 + 0.2 * torch.randn((K,), generator=g, device="cuda")).to(torch.bfloat16)
    if op == "norm_backward":
        M = case["M"]
        stream = _type(case["stream"])
        s["y"] = _normal(g, (M, K), 3.0, stream)
        s["rstd"] = torch.rsqrt(s["y"].double().square().mean(1) + EPS).to(torch.float32)
        s["w"] = (1.0 + 0.2 * torch.randn((K,), generator=g, device="cuda")).to(torch.bfloat16)
        s["dh"] = _normal(g, (M, K), 0.1)
        s["dy"] = _normal(g, (M, K), 0.1, stream)
    if op in ("norm_i8", "gemm", "experts"):
        N, G = case["N"], case["G"]
        shape = (case["E"], N) if op == "experts" else (N,)
        s["packed"], s["scales"] = _packed(g, shape, K, G)
        if case["bias"]:
            s["bias"] = _normal(g, shape, 0.1)
        T = case["tokens"] * case["top"] if op == "experts" else case["M"]
        if op == "experts":
            rows, s["offsets"] = _routes(g, case)
            if case["gather"]:
                s["rows"] = rows
        if op != "norm_i8":
            s["q"], s["qs"] = _rows_i8(g, case["tokens"] if "rows" in s else T, K)
        if case["residual"]:
            s["res"] = _normal(g, (T, N), 1.0, _type(case["out"]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "experts":
        s["ends"] = s["offsets"].tolist()        # a program that loops over experts has them on the host
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
    if c["op"] == "norm":
        return tq.rms_norm_forward(s["x"], s["w"], s.get("r"), eps=EPS)               # h, y, rstd
    if c["op"] == "norm_backward":
        return tq.rms_norm_backward(s["dh"], s["y"], s["rstd"], s["w"], dy=s["dy"])   # dx, dw
    epilogue = dict(bias=s.get("bias"), act=None if c["act"] == "none" else c["act"], residual=s.get("res"),
                    dtype=_type(c["out"]))
    if c["op"] == "norm_i8":
        q, qs, y = tq.rms_norm_i8(s["x"], s["w"], s["r"], eps=EPS)
        return tq.gemm_i8(q, qs, s["packed"], s["scales"], c["N"], c["K"], c["G"], **epilogue), y, qs
    if c["op"] == "gemm":
        return tq.gemm_i8(s["q"], s["qs"], s["packed"], s["scales"], c["N"], c["K"], c["G"], **epilogue)
    return tq.expert_gemm_i8(s["q"], s["qs"], s["packed"], s["scales"], s["offsets"], c["N"], c["K"], c["G"],
                             rows=s.get("rows"), **epilogue)


def _quantized(x, r, w):
    """(codes of each row, their scale, the sum, 1 / rms): the codes in 64 bits, since they round at borders."""
    y = x if r is None else (x.to(torch.float32) + r.to(torch.float32)).to(r.dtype)
    y64 = y.to(torch.float64)
    rstd = 1.0 / torch.sqrt((y64 * y64).mean(1) + EPS)
    t = y64 * w.to(torch.float64)
    top = t.abs().amax(1)
    q = torch.round(127.0 * t / top[:, None])
    return q, (top * rstd / 127.0).to(torch.float32), y, rstd.to(torch.float32)


def _unpack(packed, scales, N, K, G):
    nG, B = K // G, _GROUP_BYTES[G]
    p = packed.view(N, nG, B, 1).to(torch.int16)
    powers = torch.tensor([1, 3, 9, 27, 81], dtype=torch.int16, device=packed.device)
    digit = torch.remainder(torch.div(p, powers, rounding_mode="floor"), 3)
    code = digit.view(N, nG, 5 * B)[:, :, :G].to(torch.float32) - 1.0
    return (code * scales.view(N, nG, 1).to(torch.float32)).view(N, K)


def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "relu2":
        return torch.where(v > 0, v * v, torch.zeros_like(v))
    return v


def _product(q, qs, packed, scales, bias, c):
    x = q.to(torch.float32) * qs[:, None]
    v = x @ _unpack(packed, scales, c["N"], c["K"], c["G"]).t()
    return _act(v if bias is None else v + bias.to(torch.float32), c["act"])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        q, qs, y, rstd = _quantized(s["x"], s.get("r"), s["w"])
        return (q.to(torch.float32) * qs[:, None]).to(torch.bfloat16), y, rstd
    if c["op"] == "norm_backward":
        rstd = s["rstd"][:, None]
        n = s["y"].to(torch.float32) * rstd
        dh = s["dh"].to(torch.float32)
        dn = dh * s["w"].to(torch.float32)
        dx = rstd * (dn - n * (dn * n).mean(1, keepdim=True)) + s["dy"].to(torch.float32)
        return dx.to(s["y"].dtype), (dh * n).sum(0).to(s["w"].dtype)
    more = ()
    if c["op"] == "norm_i8":
        q, qs, y, _ = _quantized(s["x"], s["r"], s["w"])
        more = (y, qs)
    else:
        q, qs = s["q"], s["qs"]
    bias = s.get("bias")
    if c["op"] == "experts":
        if "rows" in s:
            q, qs = q[s["rows"]], qs[s["rows"]]
        ends = s["ends"]
        v = torch.cat([_product(q[a:b], qs[a:b], s["packed"][e], s["scales"][e], None if bias is None else bias[e], c)
                       for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a])
    else:
        v = _product(q, qs, s["packed"], s["scales"], bias, c)
    if "res" in s:
        v = v + s["res"].to(torch.float32)
    v = v.to(_type(c["out"]))
    return (v, *more) if more else v


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    K, op = case["K"], case["op"]
    wide = 2 if case.get("stream", "bf16") == "bf16" else 4
    if op == "norm":
        M = case["M"]
        # x, the stream and the sum, h; the weights and 1 / rms
        each = 2 + wide + wide + 2 if case["residual"] else wide + 2
        return {"bytes": M * K * each + 2 * K + 4 * M, "flops": 8 * M * K}
    if op == "norm_backward":
        M = case["M"]
        return {"bytes": M * K * (2 + 3 * wide) + 4 * K + 4 * M, "flops": 10 * M * K}
    N, G = case["N"], case["G"]
    weights = N * (K // G) * (_GROUP_BYTES[G] + 2)
    T = case["tokens"] * case["top"] if op == "experts" else case["M"]
    size = 2 if case["out"] == "bf16" else 4
    used = min(case["E"], T) if op == "experts" else 1
    rows = case["tokens"] if op == "experts" and case["gather"] else T
    inputs = 6 * T * K if op == "norm_i8" else rows * (K + 4)
    out = T * N * size * (2 if case["residual"] else 1)
    return {"bytes": used * (weights + (2 * N if case["bias"] else 0)) + inputs + out, "flops": 2 * T * N * K}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _weights64(packed, scales, N, K, G):
    """Every byte value's five digits looked up, times the group's scale."""
    table = torch.tensor([[v // 3 ** i % 3 - 1 for i in range(5)] for v in range(243)],
                         dtype=torch.int8, device=packed.device)
    rows = table[packed.reshape(-1).to(torch.int32)].view(N * (K // G), -1)[:, :G]
    return (rows.to(torch.float64) * scales.to(torch.float64).reshape(-1, 1)).view(N, K)


def _act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.sigmoid((8 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    return v.clamp(min=0) ** 2 if act == "relu2" else v


def exact(case, seed):
    s = _inputs(case, seed)
    op, c = case["op"], case
    if op == "norm_backward":
        y, w, dh = s["y"].double(), s["w"].double(), s["dh"].double()
        r = s["rstd"].double()[:, None]
        K = y.shape[1]
        along = torch.einsum("mk,mk,k->m", dh, y, w)[:, None]
        dx = r * dh * w - y * (r ** 3 / K) * along + s["dy"].double()
        return dx, torch.mv((y * dh).t().contiguous(), r[:, 0])
    if op in ("norm", "norm_i8"):
        total = s["x"].double() + (s["r"].double() if "r" in s else 0.0)
        # the stream is what its type holds of the sum, and that is what is normalized
        y = total.to(s["r"].dtype).double() if "r" in s else total
        rms = (y.pow(2).sum(1) / y.shape[1] + EPS).sqrt()
        h = y * s["w"].double()
        peak = h.abs().max(1).values[:, None]
        codes = (h / peak * 127).round()
        scale = peak[:, 0] / rms / 127
        if op == "norm":
            return codes * scale[:, None], total, 1 / rms
        x = codes * scale[:, None]
    else:
        x = s["q"].double() * s["qs"].double()[:, None]
    N, K, G = c["N"], c["K"], c["G"]
    if op == "experts":
        if c["gather"]:
            x = x.index_select(0, s["rows"].long())
        v = torch.empty((x.shape[0], N), dtype=torch.float64, device=x.device)
        at = s["offsets"].tolist()
        for e in range(c["E"]):
            if at[e] < at[e + 1]:
                part = torch.mm(x[at[e]:at[e + 1]], _weights64(s["packed"][e], s["scales"][e], N, K, G).t())
                v[at[e]:at[e + 1]] = part + (s["bias"][e].double() if c["bias"] else 0.0)
    else:
        v = torch.mm(x, _weights64(s["packed"], s["scales"], N, K, G).t())
        if c["bias"]:
            v = v + s["bias"].double()
    v = _act64(v, c["act"])
    if c["residual"]:
        v = v + s["res"].double()
    return (v, total, scale) if op == "norm_i8" else v

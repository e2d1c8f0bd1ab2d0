"""Float64 references of the norm into 8-bit rows and of the products that read
them, with the error bounds their tests use, and seeded inputs.

Bounds.  Codes are exact: t = y w has at most 32 bits where one of the two is
bf16, so 127 t / top differs from a border by at least 2^-40 of itself or not at
all, and float64 rounds it to the right side.  A float32 sum of squares passes
through at most 16 terms a thread and ten additions between threads (26 2^-24
relative, half of that in 1 / rms), and a few operations follow: 2^-19.
A product's sum over nG groups in float32 is off by at most nG 2^-24 times the
sum of magnitudes, whatever its order; 2^-23 covers the scale's product as well.
An activation is evaluated from a handful of float32 operations: 2^-18 of its
argument's scale.  A rounding to type t is off by finfo(t).eps / 2 relative."""
import numpy as np
import torch

from tests import ffn_reference as ref

ROW = 2.0 ** -19
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


def norm64(x, r, w, eps):
    """(codes, scale, 1 / rms, y): y as stored, codes and the rest in float64."""
    y = x if r is None else (x.float() + r.float()).to(r.dtype)
    y64 = y.double()
    rstd = 1.0 / (y64.pow(2).mean(1) + eps).sqrt()
    t = y64 if w is None else y64 * w.double()
    top = t.abs().amax(1)
    q = torch.from_numpy(np.rint((127.0 * t / torch.where(top > 0, top, torch.ones_like(top))[:, None]).numpy()))
    return q, top * rstd / 127.0, rstd, y


def norm_back64(dh, y, rstd, w, dy):
    """((dx, its bound), (dw, its bound)) before the roundings to their types."""
    n, r = y.double() * rstd.double()[:, None], rstd.double()[:, None]
    dn = dh.double() if w is None else dh.double() * w.double()
    dx = r * (dn - n * (dn * n).mean(1, keepdim=True))
    size = r * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    if dy is not None:
        dx, size = dx + dy.double(), size + dy.double().abs()
    # a thread's 24 terms at most and ten additions; dw: at most 100 in a row
    return (dx, 2.0 ** -18 * size), ((dh.double() * n).sum(0), 2.0 ** -17 * (dh.double() * n).abs().sum(0))


def activate64(v, act):
    """(act(v), the largest |act'| near v)."""
    if act in ("silu", "gelu"):
        return ref.gate64(v, act)[0], torch.full_like(v, 1.13)
    if act == "relu2":
        return v.clamp(min=0) ** 2, 2 * v.abs()
    return v, torch.ones_like(v)


def product64(q, qs, packed, scales, N, K, G, bias=None, act=None, residual=None, out=torch.bfloat16):
    """(result, bound of an error of the rounded result)."""
    w = ref.weight64(packed, scales, N, K, G).view(N, K // G, G)
    x = q.double().view(q.shape[0], K // G, G)
    parts = torch.einsum("mgj,ngj->mng", x, w) * qs.double()[:, None, None]
    v, size = parts.sum(-1), parts.abs().sum(-1)
    if bias is not None:
        v, size = v + bias.double(), size + bias.double().abs()
    off = (K // G + 4) * ref.ACC * size
    y, slope = activate64(v, act)
    off = slope * off + off * off + (ref.EVAL * size + ref.ACC * y.abs() if act else 0.0)
    if residual is not None:
        y = y + residual.double()
        off = off + 2.0 ** -24 * (y.abs() + residual.double().abs())
    return y, off * (1 + 2.0 ** -7) + half_step(out) * y.abs() + 2.0 ** -130


def rows_i8(seed, M, K):
    """Random 8-bit rows (-128 among them) and scales."""
    rng = np.random.default_rng(seed)
    q = np.clip(np.rint(rng.standard_normal((M, K)) * 40), -128, 127).astype(np.int8)
    q[rng.random((M, K)) < 0.002] = -128
    return torch.from_numpy(q), torch.from_numpy((0.02 * np.exp(0.3 * rng.standard_normal(M))).astype(np.float32))


def within(got, want, bound, what):
    err = (got.detach().cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d off; first at %s: %r, not %r, bound %.3g" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got.cpu()[bad][0].item(),
        want[bad][0].item(), (bound if torch.is_tensor(bound) else torch.full_like(want, bound))[bad][0].item())


# (rows, N, K, G, experts or 0): together they reach every kernel of the products,
# with and without splits of K, in one round of tiles and more (tests/test_i8_plans.py
# sees to it)
MIDDLE = [(3, 40, 192, 64, 0), (2, 9000, 4096, 64, 0), (4, 3000, 2048, 64, 0), (7, 40, 128, 64, 0), (6, 80, 14336, 64, 0), (14, 70, 448, 64, 0),
          (15, 300, 4032, 64, 0), (2, 33, 384, 128, 0), (1, 2000, 8192, 128, 0), (8, 50, 640, 128, 0),
          (5, 17, 7168, 128, 0), (13, 200, 1024, 128, 0), (16, 130, 5760, 128, 0), (30, 77, 192, 64, 0),
          (40, 140, 1088, 64, 0), (50, 260, 128, 128, 0), (65, 130, 2176, 128, 0), (20, 48, 320, 64, 9),
          (40, 600, 2048, 64, 16), (9, 40, 256, 128, 3), (64, 1000, 2048, 128, 16), (70, 90, 640, 128, 3),
          (16, 70000, 576, 64, 0), (16, 70000, 640, 128, 0), (7, 280000, 128, 128, 0), (6, 280000, 64, 64, 0),
          (3, 280000, 128, 64, 0), (4, 280000, 128, 128, 0), (16, 60000, 64, 64, 0), (16, 60000, 128, 128, 0)]
LARGE = [(771, 5000, 64, 64, 0), (986, 2600, 192, 64, 20), (2286, 513, 4224, 64, 0), (1608, 513, 5504, 64, 20),
         (3113, 2600, 64, 64, 0), (2694, 2600, 320, 64, 20), (1677, 5000, 3520, 64, 1),
         (778, 5000, 128, 128, 0), (976, 2600, 384, 128, 20), (1350, 1024, 4992, 128, 0), (963, 1500, 4224, 128, 1),
         (3099, 2600, 128, 128, 0), (3113, 2597, 384, 128, 0), (2628, 2600, 1024, 128, 20),
         (3093, 2600, 9600, 128, 0), (1721, 5000, 3840, 128, 1),
         (964, 4100, 5376, 128, 0), (1476, 2600, 5632, 128, 5), (2061, 2000, 6016, 128, 2),
         (700, 6000, 192, 64, 20), (700, 6000, 128, 128, 20), (3099, 8200, 256, 128, 0),
         (1500, 6000, 128, 128, 20), (1500, 6000, 192, 64, 20), (3000, 6000, 192, 64, 10)]


def segments(rng, E, T):
    """Uneven segments, some empty, with rows of none before and behind."""
    cuts = np.sort(rng.integers(T // 20, T - T // 20 + 1, E + 1)) if E > 1 else np.array([T // 50, T - T // 70])
    return cuts.astype(np.int32)

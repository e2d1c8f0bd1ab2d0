"""Float64 references of the gated feed-forward and adapter operators, with
the error bounds their tests use, and seeded inputs for them.

Bounds.  A kernel's products are exact in fp32 (bf16 times a ternary code or
bf16) and its sums are fp32: a sum of n terms in any order is off by at most
n 2^-24 times the sum of magnitudes; 2^-23 is used, which also covers the
group scale's product.  A rounding to bf16 adds half a unit in the last
place: at most 2^-8 relative (at the bottom of a binade), 0.0017 < 2^-9 in root
mean square over many values.  act and act' are evaluated in fp32 from a handful of operations: 2^-18
of their arguments' scale covers them (|act'| <= 1.13).
"""
import math

import numpy as np
import torch

_DIGITS = np.array([[v // 3 ** i % 3 - 1 for i in range(5)] for v in range(243)], np.int8)
ACC = 2.0 ** -23
EVAL = 2.0 ** -18


def packed_weight(seed, N, K, G, scale=0.02, zero_groups=0.05):
    """Random packed codes (valid padding) and fp16 scales, some of them 0:
    uint8 [N, K/G * B], fp16 [N, K/G] host tensors."""
    rng = np.random.default_rng(seed)
    nG, B = K // G, (G + 4) // 5
    d = rng.integers(0, 3, size=(N, nG, 5 * B)).astype(np.uint8)
    d[:, :, G:] = 1
    p = (d.reshape(N, nG, B, 5) * np.array([1, 3, 9, 27, 81], np.uint8)).sum(-1).astype(np.uint8)
    s = (scale * np.exp(0.3 * rng.standard_normal((N, nG)))).astype(np.float16)
    s[rng.random((N, nG)) < zero_groups] = 0
    return torch.from_numpy(p.reshape(N, nG * B)), torch.from_numpy(s)


def weight64(packed, scales, N, K, G):
    c = _DIGITS[packed.numpy()].reshape(N, K // G, -1)[:, :, :G].astype(np.float64)
    return torch.from_numpy((c * scales.numpy().astype(np.float64)[:, :, None]).reshape(N, K))


def normal(seed, shape, sigma=1.0, dtype=torch.bfloat16):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).to(dtype)


def gate64(g, act):
    """(act(g), act'(g)) in float64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)


def glu64(x, wg, wu, act):
    """h, g, u in float64 and the bound on an error of h before its rounding."""
    K = x.shape[1]
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = K * ACC * (x.abs() @ wg.abs().t()), K * ACC * (x.abs() @ wu.abs().t())
    a = gate64(g, act)[0]
    pre = (1.13 * eg + EVAL * g.abs()) * (u.abs() + eu) + a.abs() * eu
    return a * u, g, u, pre, eg, eu


def check(got, want, pre, what, bf16=True):
    """|got - want| <= pre + the rounding, every element; and, so that a small
    systematic error does not hide under the bound, the root mean square of
    the error over many values is at most that of the roundings plus the
    bound's."""
    got, pre = got.double().cpu(), pre + 1e-38
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    tol = pre + want.abs() * (2.0 ** -8 if bf16 else ACC)
    err = (got - want).abs()
    if (err > tol).any():
        i = tuple(((err - tol) == (err - tol).max()).nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d outside; worst at %s: got %r want %r tol %r" % (
            what, int((err > tol).sum()), err.numel(), i, got[i].item(), want[i].item(), tol[i].item()))
    if bf16 and want.numel() >= 1024:
        rms = lambda t: float(t.square().mean().sqrt())  # noqa: E731
        assert rms(err) <= 2.0 ** -9 * rms(want) + rms(pre), (what, rms(err), rms(want))


def lora64(x, w, ids, a, b, scaling):
    """y in float64 and the bound on its error."""
    K, R = x.shape[1], a.shape[1] if a.numel() else 0
    y, bound = x @ w.t(), K * ACC * (x.abs() @ w.abs().t())
    for i, q in enumerate(ids.tolist()):
        if 0 <= q < a.shape[0]:
            t, ta = a[q] @ x[i], a[q].abs() @ x[i].abs()
            y[i] += scaling[q] * (b[q] @ t)
            bound[i] += (K + R + 2) * ACC * scaling[q].abs() * (b[q].abs() @ ta)
    return y, bound


def backward64(dh, x, wg, wu, g, u, act):
    """(dx, dwg, dwu) in float64 and their error bounds before the final
    rounding: dg and du are rounded to bf16 on the way to the products."""
    a, slope = gate64(g, act)
    dg, du = dh * u * slope, dh * a
    edg = 2.0 ** -8 * dg.abs() + 2 * EVAL * (dh * u).abs() * (1 + g.abs())
    edu = 2.0 ** -8 * du.abs() + 2 * EVAL * (dh * g).abs()
    M, N = dh.shape
    n = 2 * N * ACC
    pdx = edg @ wg.abs() + edu @ wu.abs() + n * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    m = M * ACC
    pg = edg.t() @ x.abs() + m * (dg.abs().t() @ x.abs())
    pu = edu.t() @ x.abs() + m * (du.abs().t() @ x.abs())
    return (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x), (pdx, pg, pu)

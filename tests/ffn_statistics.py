"""Root-mean-square checks beside the worst-case bounds of ffn_reference.

The worst case of an fp32 sum of n terms is n 2^-24 of the sum of their
magnitudes, which for long sums is far above what any sum does: a result that
lacks a whole stage of K can lie below it.  Rounding errors are independent
enough to add in squares: adding a term to a running sum s is off by up to
2^-24 |s|, and the running sums of n terms of either sign with root mean square
q are about q sqrt(i) for i = 1 .. n, so the error's root mean square is at most
2^-24 q n / sqrt(6) = 0.41 * 2^-24 sqrt(n) S with S^2 the sum of the terms'
squares.  2^-24 (sqrt(n) + 2) S is used: more than twice that, and a rounding or
two of the result.  A rounding to bf16 is off by a value even in +-u / 2, u the
unit in the last place (2^-7 of the binade's lower end): its square is u^2 / 12
in the mean, with a variance of u^4 / 180; six deviations of their mean over
the values checked are allowed.
"""
import torch

UNIT = 2.0 ** -24


def rms(t):
    return float(t.square().mean().sqrt())


def rounding(want):
    """What roundings to bf16 of these values may add up to, root mean square."""
    u = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(1e-38))) - 7)
    mean = u.square().mean() / 12 + 6 * (u.square().square().sum() / 180).sqrt() / u.numel()
    return float(mean.sqrt())


def of_product(x, w):
    """The deviation of each element of x w^T summed in fp32 (float64 x [M,K],
    w [N,K])."""
    return UNIT * (x.shape[1] ** 0.5 + 2) * (x.square() @ w.square().t()).sqrt()


def of_adapters(x, ids, a, b, scaling):
    """That of the adapters' part alone: t in fp32 (24 bits), then its product
    with B."""
    K, R = x.shape[1], a.shape[1]
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64, device=x.device)
    for i in range(a.shape[0]):
        at = (ids.to(x.device) == i).nonzero()[:, 0]
        if len(at):
            t = x[at] @ a[i].t()
            dev = (K ** 0.5 + 2) * (x[at].square() @ a[i].square().t()).sqrt()
            out[at] = scaling[i].abs() * UNIT * (((dev.square() @ b[i].square().t()).sqrt())
                                                 + (R ** 0.5 + 4) * (t.square() @ b[i].square().t()).sqrt())
    return out


def check_rms(got, want, deviation, what, bf16):
    """The root mean square of the error, over all the elements and over each
    sixteenth of the rows and of the columns, is at most that of the deviations
    and of the result's own rounding.  A block of fewer than 256 elements is
    left to the worst-case bound."""
    got, want, deviation = (t.to(torch.float64).to(want.device) for t in (got, want, deviation))
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = got - want
    blocks = [(err, want, deviation)]
    for dim in (0, 1):
        step = max(1, want.shape[dim] // 16)
        blocks += list(zip(*(t.split(step, dim) for t in (err, want, deviation))))
    for e, w, d in blocks:
        if e.numel() < 256:
            continue
        limit = (rounding(w) if bf16 else 0.0) + rms(d) + 1e-38
        assert rms(e) <= limit, "%s: error %.3g, at most %.3g (values %.3g)" % (what, rms(e), limit, rms(w))


def rounded_gates(dh, g, u, gate):
    """(dg, du) as the backward call holds them: rounded once to bf16."""
    a, slope = gate
    return ((dh * u * slope).to(torch.bfloat16).double(), (dh * a).to(torch.bfloat16).double())

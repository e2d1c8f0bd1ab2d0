"""The checks of ffn_statistics pass results with the rounding errors of fp32
sums and reject the mistakes that the worst-case bounds of ffn_reference let
through.  On the CPU; every mistake is planted in the values checked."""
import pytest
import torch

from tests import ffn_reference as ref
from tests import ffn_statistics as stat


def _glu(M, N, K, G):
    x, gate, up = ref.normal(3, (M, K)), ref.packed_weight(5, N, K, G), ref.packed_weight(6, N, K, G)
    return x, ref.weight64(*gate, N, K, G), ref.weight64(*up, N, K, G)


def _fp32(x, w, keep=None):
    """x w^T in fp32, 32 k after another; the stages in `keep` alone."""
    y = torch.zeros(x.shape[0], w.shape[0])
    x, w = x.float(), w.float()
    for k in range(0, x.shape[1], 32):
        if keep is None or keep(k):
            y += x[:, k:k + 32] @ w[:, k:k + 32].t()
    return y


@pytest.mark.parametrize("M,N,K,G", [(70, 64, 33024, 128), (64, 96, 16448, 64), (90, 60, 7296, 64), (100, 80, 640, 64)])
def test_gated_block(M, N, K, G):
    x, wg, wu = _glu(M, N, K, G)
    want, g, u, pre, _, _ = ref.glu64(x.double(), wg, wu, "silu")
    dev = 1.13 * stat.of_product(x.double(), wg) * u.abs() + g.abs() * stat.of_product(x.double(), wu)

    def h(keep=None, keep_up=None):
        a, b = _fp32(x, wg, keep), _fp32(x, wu, keep_up)
        return (torch.nn.functional.silu(a) * b).to(torch.bfloat16)

    stat.check_rms(h(), want, dev, "fp32", True)
    ref.check(h(), want, pre, "fp32")
    for wrong in (h(keep=lambda k: k != K // 64 * 32), h(keep_up=lambda k: k < K - 32), h() * 0.99,
                  h(keep=lambda k: k < K - 512 or K < 1024, keep_up=lambda k: k < K - 512 or K < 1024) if K > 1024 else h() * 1.01):
        with pytest.raises(AssertionError):
            stat.check_rms(wrong, want, dev, "mistake", True)


@pytest.mark.parametrize("M,N,K,G,R", [(32, 70, 14336, 128, 16), (40, 60, 17408, 128, 40), (60, 50, 2176, 64, 64),
                                       (64, 40, 16512, 128, 8)])
def test_adapters(M, N, K, G, R):
    n = 3
    x, w = ref.normal(3, (M, K)), ref.packed_weight(5, N, K, G)
    w = ref.weight64(*w, N, K, G)
    a, b = ref.normal(7, (n, R, K), K ** -0.5), ref.normal(8, (n, N, R), 0.3)
    scaling, ids = torch.tensor([1.0, -0.5, 2.0]), torch.arange(M, dtype=torch.int32) % n
    d = (x.double(), w, ids, a.double(), b.double(), scaling.double())
    want, bound = ref.lora64(*d)
    part, _ = ref.lora64(d[0], w * 0, *d[2:])
    dev_part = stat.of_adapters(d[0], ids, *d[3:])
    dev = (dev_part.square() + stat.of_product(d[0], w).square()).sqrt()

    def y(projection, change=lambda t: t, keep=None):
        out = _fp32(x, w) if projection else torch.zeros(M, N)
        for i in range(n):
            at = ids == i
            out[at] += _fp32(change(_fp32(x[at], a[i], keep)), b[i]) * scaling[i]
        return out

    stat.check_rms(y(True), want, dev, "fp32", False)
    stat.check_rms(y(False), part, dev_part, "fp32", False)
    ref.check(y(True), want, bound, "fp32", bf16=False)
    mistakes = [dict(change=lambda t: t * 0.98), dict(change=lambda t: t.to(torch.bfloat16).float()),
                dict(keep=lambda k: k != 64), dict(change=lambda t: t * (1 + 2.0 ** -15))]
    for m in mistakes:
        with pytest.raises(AssertionError):
            stat.check_rms(y(False, **m), part, dev_part, "mistake", False)
    for m in mistakes[:3]:
        with pytest.raises(AssertionError):
            stat.check_rms(y(True, **m), want, dev, "mistake", False)


def test_gradients():
    """Gradients from dg and du in bf16 pass against those same roundings in
    64 bits; a missing stage, one weight matrix alone or unrounded dg do not."""
    M, N, K = 96, 160, 128
    x, wg, wu = ref.normal(3, (M, K)).double(), ref.normal(4, (N, K), 0.05).double(), ref.normal(5, (N, K), 0.05).double()
    g, u, dh = (x @ wg.t()).to(torch.bfloat16).double(), (x @ wu.t()).to(torch.bfloat16).double(), ref.normal(6, (M, N)).double()
    gate = ref.gate64(g, "silu")
    dg, du = stat.rounded_gates(dh, g, u, gate)
    both, w = torch.cat([dg, du], 1), torch.cat([wg, wu])
    want, dev = both @ w, stat.of_product(both, w.t().contiguous())
    stat.check_rms(_fp32(both, w.t()).to(torch.bfloat16), want, dev, "dx", True)
    for wrong in (_fp32(both, w.t(), lambda k: k != 288), _fp32(dg, wg.t()),
                  _fp32(torch.cat([dh * u * gate[1], dh * gate[0]], 1), w.t())):
        with pytest.raises(AssertionError):
            stat.check_rms(wrong.to(torch.bfloat16), want, dev, "mistake", True)

"""RMSNorm as autograd sees it, on the CPU: its two calls are replaced by the
formulas in torch, so no kernel is launched."""
import pytest
import torch

import ternary_weight_only_amd as tq
from ternary_weight_only_amd import binding
from tests import ffn_reference as ref

EPS = 1e-6


@pytest.fixture
def stand_ins(monkeypatch):
    """rms_norm_forward and rms_norm_backward in float64, without the rounding to
    8 bits."""
    def forward(x, weight=None, residual=None, eps=EPS, status=None, out=None):
        y = x if residual is None else x + residual
        rstd = 1 / (y.square().mean(1) + eps).sqrt()
        n = y * rstd[:, None]
        return n if weight is None else n * weight, y, rstd

    def backward(dh, y, rstd, weight=None, dy=None, out=None, workspace=None):
        n, r = y * rstd[:, None], rstd[:, None]
        dn = dh if weight is None else dh * weight
        dx = r * (dn - n * (dn * n).mean(1, keepdim=True))
        return dx if dy is None else dx + dy, None if weight is None else (dh * n).sum(0)

    monkeypatch.setattr(binding, "rms_norm_forward", forward)
    monkeypatch.setattr(binding, "rms_norm_backward", backward)


def _leaves():
    return [ref.normal(3 + i, s, 1.0, torch.float64).requires_grad_() for i, s in enumerate(((5, 64), (64,), (5, 64)))]


@pytest.mark.parametrize("of", ["x", "weight", "residual", "dh"])
def test_a_second_gradient_raises_and_names_the_operator(stand_ins, of):
    x, w, r = _leaves()
    dh = torch.ones(5, 64, dtype=torch.float64, requires_grad=of == "dh")
    h, y = tq.RMSNorm.apply(x, w, r)
    grads = torch.autograd.grad(h, (x, w, r), dh, create_graph=True)
    with pytest.raises(tq.TQError, match="^RMSNorm has no gradients of gradients"):
        torch.autograd.grad(sum(g.square().sum() for g in grads), {"x": x, "weight": w, "residual": r, "dh": dh}[of])


def test_a_second_gradient_of_the_gated_block_names_it(monkeypatch):
    monkeypatch.setattr(binding, "glu_forward", lambda x, wg, wu, act: ref.glu64(x, wg, wu, act)[:3])
    monkeypatch.setattr(binding, "glu_backward", lambda dh, x, wg, wu, g, u, act: ref.backward64(dh, x, wg, wu, g, u, act)[0])
    leaves = [ref.normal(i, s, 1.0, torch.float64).requires_grad_() for i, s in enumerate(((5, 64), (8, 64), (8, 64)))]
    (g, *_) = torch.autograd.grad(tq.GLU.apply(*leaves).sum(), leaves, create_graph=True)
    with pytest.raises(tq.TQError, match="^GLU has no gradients of gradients"):
        torch.autograd.grad(g.square().sum(), leaves[0])

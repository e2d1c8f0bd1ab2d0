"""GLU as autograd sees it, on the CPU: its two calls are replaced by the
formulas in torch, so no kernel is launched."""
import pytest
import torch

import ternary_weight_only_amd as tq
from ternary_weight_only_amd import binding
from tests import ffn_reference as ref


@pytest.fixture
def stand_ins(monkeypatch):
    """glu_forward and glu_backward in float64; the list of the dh that the
    backward call received, with the list `saved` of the forward calls' save."""
    class Received(list):
        pass

    received = Received()
    received.saved = []

    def forward(x, wg, wu, act="silu", save=True, out=None):
        received.saved.append(save)
        h, g, u, _, _, _ = ref.glu64(x, wg, wu, act)
        return (h, g, u) if save else h

    def backward(dh, x, wg, wu, g, u, act="silu", out=None, workspace=None):
        received.append(dh)
        return ref.backward64(dh, x, wg, wu, g, u, act)[0]

    monkeypatch.setattr(binding, "glu_forward", forward)
    monkeypatch.setattr(binding, "glu_backward", backward)
    return received


def _leaves():
    return [ref.normal(3 + i, s, 1.0, torch.float64).requires_grad_() for i, s in enumerate(((5, 64), (8, 64), (8, 64)))]


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_first_gradients(stand_ins, act):
    leaves = _leaves()
    assert torch.autograd.gradcheck(lambda *t: tq.GLU.apply(*t, act), leaves)


@pytest.mark.parametrize("of", [0, 1, 2, None])
@pytest.mark.parametrize("to", [0, 1, 2])
def test_a_second_gradient_raises(stand_ins, of, to):
    """The backward call's results carry no graph: a gradient through them
    would be dropped without a word.  First gradients with create_graph are
    those without."""
    leaves = _leaves()
    dh = torch.ones(5, 8, dtype=torch.float64, requires_grad=of is None)
    want = torch.autograd.grad(tq.GLU.apply(*leaves), leaves, dh.detach())
    h = tq.GLU.apply(*leaves)
    got = torch.autograd.grad(h, leaves, dh, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(tq.TQError, match="gradients of gradients"):
        second = got[of or 0].square().sum() + h.sum()
        torch.autograd.grad(second, leaves[to] if of is not None else dh)


def test_a_gradient_that_starts_anywhere(stand_ins):
    """h's gradient may be rows inside a larger tensor, as the backward of cat
    makes it: the call gets it contiguous and on 16 bytes."""
    x, (wg, wu) = ref.normal(3, (5, 64)), (ref.normal(i, (13, 64)).requires_grad_() for i in (4, 5))
    whole = ref.normal(7, (8, 13))
    for rows in (whole[3:], whole[::2][:3], whole.t()[:5, :]):
        h = tq.GLU.apply(x[:rows.shape[0]], wg[:rows.shape[1]], wu[:rows.shape[1]])
        h.backward(rows)
    torch.cat([whole[:3], tq.GLU.apply(x, wg, wu)]).float().square().sum().backward()
    assert len(stand_ins) == 4
    for dh in stand_ins:
        assert dh.is_contiguous() and dh.data_ptr() % 16 == 0


def test_nothing_is_saved_where_no_gradient_can_be_asked_for(stand_ins):
    x, wg, wu = _leaves()
    want = tq.GLU.apply(x, wg, wu, "gelu")
    with torch.no_grad():
        a = tq.GLU.apply(x, wg, wu, "gelu")
    b = tq.GLU.apply(x.detach(), wg.detach(), wu.detach(), act="gelu")
    c = tq.GLU.apply(x.detach(), wg, wu.detach(), "gelu")
    assert stand_ins.saved == [True, False, False, True]
    assert want.requires_grad and c.requires_grad and not a.requires_grad and not b.requires_grad
    assert all(torch.equal(t, want) for t in (a, b, c))

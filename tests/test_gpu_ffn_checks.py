"""The binding refuses wrong shapes, types, devices and strides of the gated
feed-forward and adapter calls before any launch, and writes nothing."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref

pytestmark = pytest.mark.gpu

M, N, K, G, R, n = 6, 48, 128, 64, 8, 2


def _all():
    x = ref.normal(1, (M, K)).cuda()
    gate = tuple(t.cuda() for t in ref.packed_weight(2, N, K, G))
    up = tuple(t.cuda() for t in ref.packed_weight(3, N, K, G))
    lo = dict(ids=torch.zeros(M, dtype=torch.int32, device="cuda"),
              a=ref.normal(4, (n, R, K)).cuda(), b=ref.normal(5, (n, N, R)).cuda(),
              scaling=torch.ones(n, device="cuda"))
    w = [ref.normal(6 + i, (N, K)).cuda() for i in range(2)]
    mn = [ref.normal(8 + i, (M, N)).cuda() for i in range(3)]
    return x, gate, up, lo, w, mn


def _refused(call):
    with pytest.raises(tq.TQError):
        call()


def test_glu():
    x, gate, up, _, _, _ = _all()
    for bad in (x.float(), x[:, :64], x[:, ::2], x[0], x.cpu(), x.t()):
        _refused(lambda: tq.glu(bad, gate, up, N, K, G))
    for pair in ((gate[0][:-1], gate[1]), (gate[0], gate[1][:-1]), (gate[0].cpu(), gate[1]),
                 (gate[0], gate[1].float()), (gate[0].to(torch.int8), gate[1])):
        _refused(lambda: tq.glu(x, pair, up, N, K, G))
        _refused(lambda: tq.glu(x, gate, pair, N, K, G))
    for act in ("relu", None, 0):
        _refused(lambda: tq.glu(x, gate, up, N, K, G, act=act))
    out = torch.full((M, N), 3.0, device="cuda")
    _refused(lambda: tq.glu(x, gate, up, N, K, G, out=out))
    _refused(lambda: tq.glu(x, gate, up, N, K, G, out=out.bfloat16()[:-1]))
    _refused(lambda: tq.glu(x, gate, up, N, K, 32))
    _refused(lambda: tq.glu(x, gate, up, N, K, G, workspace=torch.zeros(64)))
    assert (out == 3.0).all()
    # a view that starts off the required alignment is refused by the library
    buf = torch.zeros(M * K + 8, dtype=torch.bfloat16, device="cuda")
    _refused(lambda: tq.glu(buf[1:1 + M * K].view(M, K), gate, up, N, K, G))


def test_lora():
    x, w, _, lo, _, _ = _all()

    def call(**kw):
        a = {**lo, **kw}
        return tq.lora_matmul(a.pop("x", x), *w, a.pop("ids"), a.pop("a"), a.pop("b"),
                              a.pop("scaling"), N, K, G, **a)

    call()
    for kw in (dict(ids=lo["ids"].long()), dict(ids=lo["ids"][:-1]), dict(ids=lo["ids"].cpu()),
               dict(a=lo["a"][:1]), dict(a=lo["a"][:, :, :64]), dict(a=lo["a"].float()),
               dict(b=lo["b"][:, :-1]), dict(b=lo["b"].transpose(1, 2)), dict(b=lo["b"][:1]),
               dict(scaling=lo["scaling"].double()), dict(scaling=lo["scaling"][:1]),
               dict(a=lo["a"][:, :4].contiguous(), b=lo["b"][:, :, :4].contiguous()),
               dict(out=torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")),
               dict(workspace=torch.zeros(1, dtype=torch.uint8, device="cuda")),
               dict(status=torch.zeros(1, dtype=torch.int64, device="cuda"))):
        _refused(lambda: call(**kw))


def test_train():
    x, _, _, _, w, mn = _all()
    for bad in (w[0][:-1], w[0].float(), w[0][:, :64], w[0].t().contiguous().t(), w[0].cpu()):
        _refused(lambda: tq.glu_forward(x, w[0], bad))
        _refused(lambda: tq.glu_backward(mn[0], x, w[0], bad, mn[1], mn[2]))
    for i in range(3):
        for bad in (mn[i][:-1], mn[i].float(), mn[i].t(), mn[i].cpu()):
            t = list(mn)
            t[i] = bad
            _refused(lambda: tq.glu_backward(t[0], x, *w, t[1], t[2]))
    _refused(lambda: tq.glu_forward(x[:, :96].contiguous(), *[t[:, :96].contiguous() for t in w]))
    _refused(lambda: tq.glu_forward(x, *w, out=(mn[0], mn[1], mn[2].float())))
    _refused(lambda: tq.glu_backward(mn[0], x, *w, mn[1], mn[2], out=(x, w[0], w[1].float())))
    _refused(lambda: tq.glu_backward(mn[0], x, *w, mn[1], mn[2],
                                     workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")))

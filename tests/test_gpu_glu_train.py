"""tq_glu_forward and tq_glu_backward on the GPU against the float64 formulas,
and the gradients against differences of the loss."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _weights(seed, N, K):
    return ref.normal(seed, (N, K), 0.05), ref.normal(seed + 1, (N, K), 0.05)



SHAPES = [(1, 1, 64), (1, 8, 64), (2, 17, 128), (16, 16, 64), (33, 100, 192), (64, 64, 64),
          (75, 700, 512), (129, 257, 320), (255, 256, 256), (257, 264, 128), (300, 1000, 1024),
          (513, 130, 576), (31, 2048, 64), (1000, 24, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(M, N, K, act):
    say("glu forward", M, N, K, act)
    x, (wg, wu) = ref.normal(3, (M, K)), _weights(5, N, K)
    h, g, u = tq.glu_forward(x.cuda(), wg.cuda(), wu.cuda(), act)
    alone = tq.glu_forward(x.cuda(), wg.cuda(), wu.cuda(), act, save=False)
    torch.cuda.synchronize()
    wh, wgv, wuv, pre, eg, eu = ref.glu64(x.double(), wg.double(), wu.double(), act)
    ref.check(h, wh, pre, "h")
    ref.check(g, wgv, eg, "g")
    ref.check(u, wuv, eu, "u")
    assert torch.equal(alone, h)


def _backward_problem(seed, M, N, K):
    x, (wg, wu) = ref.normal(seed, (M, K)), _weights(seed + 1, N, K)
    g = (x.double() @ wg.double().t()).to(torch.bfloat16)
    u = (x.double() @ wu.double().t()).to(torch.bfloat16)
    return ref.normal(seed + 3, (M, N)), x, wg, wu, g, u


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(M, N, K, act):
    say("glu backward", M, N, K, act)
    p = _backward_problem(11, M, N, K)
    got = tq.glu_backward(*[t.cuda() for t in p], act)
    torch.cuda.synchronize()
    want, pre = ref.backward64(*[t.double() for t in p], act)
    for t, w, e, name in zip(got, want, pre, ("dx", "dwg", "dwu")):
        ref.check(t, w, e, "%s M=%d N=%d K=%d" % (name, M, N, K))


@pytest.mark.parametrize("M,N,K", [(512, 768, 512), (1024, 1280, 1024), (2049, 520, 704)])
def test_larger(M, N, K):
    say("glu train larger", M, N, K)
    x, (wg, wu) = ref.normal(3, (M, K)), _weights(5, N, K)
    h, g, u = tq.glu_forward(x.cuda(), wg.cuda(), wu.cuda())
    wh, wgv, wuv, pre, eg, eu = ref.glu64(x.double(), wg.double(), wu.double(), "silu")
    ref.check(h, wh, pre, "h")
    ref.check(g, wgv, eg, "g")
    ref.check(u, wuv, eu, "u")
    p = (ref.normal(9, (M, N)), x, wg, wu, g.cpu(), u.cpu())
    got = tq.glu_backward(*[t.cuda() for t in p])
    want, pre = ref.backward64(*[t.double() for t in p], "silu")
    for t, w, e, name in zip(got, want, pre, ("dx", "dwg", "dwu")):
        ref.check(t, w, e, name)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """<gradient, v> for random directions v against the central difference of
    L = sum dh * h in float64.  The kernel's gradient has rounding errors of
    about 2^-9 (output), 2^-9 (dg, du) and 2^-9 times a factor near 1 (saved g
    and u) per element, independent of v: their projection on v has a standard
    deviation below 2^-8 |gradient|; six of them are allowed, and the
    difference quotient's own error is far smaller."""
    say("glu differences", act)
    M, N, K = 40, 96, 128
    x, (wg, wu) = ref.normal(3, (M, K)), _weights(5, N, K)
    dh = ref.normal(9, (M, N))
    leaves = [t.cuda().requires_grad_() for t in (x, wg, wu)]
    h = tq.GLU.apply(*leaves, act)
    h.backward(dh.cuda())

    def loss(*t):
        return float((dh.double() * ref.glu64(*t, act)[0]).sum())

    base = [t.double() for t in (x, wg, wu)]
    for i, leaf in enumerate(leaves):
        grad = leaf.grad.double().cpu()
        assert leaf.grad.dtype == torch.bfloat16
        for s in range(3):
            v = ref.normal(100 + s, tuple(grad.shape), 1.0, torch.float64)
            eps = 1e-4 / float(v.abs().max())
            lo, hi = list(base), list(base)
            lo[i], hi[i] = base[i] - eps * v, base[i] + eps * v
            want = (loss(*hi) - loss(*lo)) / (2 * eps)
            assert abs(float((grad * v).sum()) - want) <= 6 * 2.0 ** -8 * float(grad.norm()), (i, s)


def test_straight_through_to_the_latent_weights():
    """fake_quantize -> GLU: the latent weights receive dwg and dwu unchanged,
    a step on them runs, and x's gradient uses the ternary weights."""
    say("glu straight-through")
    M, N, K, G = 50, 128, 256, 64
    lat = [ref.normal(21 + i, (N, K), 0.05).cuda().requires_grad_() for i in range(2)]
    x = ref.normal(23, (M, K)).cuda().requires_grad_()
    hat = [tq.FakeQuantize.apply(w, G) for w in lat]
    h = tq.GLU.apply(x, *hat)
    dh = ref.normal(25, (M, N)).cuda()
    h.backward(dh)
    with torch.no_grad():
        _, g, u = tq.glu_forward(x, *hat)
        dx, dwg, dwu = tq.glu_backward(dh, x, *hat, g, u)
    assert torch.equal(x.grad, dx) and torch.equal(lat[0].grad, dwg) and torch.equal(lat[1].grad, dwu)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_saturated_gates(act):
    """Gates far out on both sides and at exactly 0: values and slopes reach
    their limits without NaN."""
    say("glu saturated", act)
    M, N, K = 16, 64, 64
    _, x, wg, wu, _, u = _backward_problem(31, M, N, K)
    g = torch.linspace(-300, 300, M * N).reshape(M, N).to(torch.bfloat16)
    g[0, 0], g[0, 1], g[0, 2] = 0.0, 3e38, -3e38
    dh = ref.normal(33, (M, N))
    dh[0, 1] = 0.0                               # 3e38 itself would overflow dwu
    got = tq.glu_backward(*[t.cuda() for t in (dh, x, wg, wu, g, u)], act)
    want, pre = ref.backward64(*[t.double() for t in (dh, x, wg, wu)],
                               g.double().clamp(-1e18, 1e18), u.double(), act)
    assert all(torch.isfinite(t.float()).all() for t in got)
    keep = torch.ones(M, dtype=torch.bool)
    keep[0] = False                              # row 0 holds the extreme gates
    ref.check(got[0][keep.cuda()], want[0][keep], pre[0][keep], "dx")


def test_repeats_are_identical_on_any_stream_and_workspace():
    say("glu train repeat")
    for M, N, K in ((33, 100, 192), (600, 1000, 512)):
        p = [t.cuda() for t in _backward_problem(41, M, N, K)]
        want = tq.glu_backward(*p)
        wantf = tq.glu_forward(*p[1:4])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ws = torch.full((max(16, tq.glu_backward_workspace(M, N, K)),), 0xFF, dtype=torch.uint8,
                            device="cuda")
            got = [tq.glu_backward(*p, workspace=ws) for _ in range(2)]
            gotf = [tq.glu_forward(*p[1:4]) for _ in range(2)]
        side.synchronize()
        for results, first in ((got, want), (gotf, wantf)):
            for r in results:
                assert all(torch.equal(a, b) for a, b in zip(r, first))


def test_no_rows():
    wg, wu = (t.cuda() for t in _weights(51, 40, 64))
    e = lambda n: torch.zeros((0, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, g, u = tq.glu_forward(e(64), wg, wu)
    assert h.shape == g.shape == u.shape == (0, 40)
    out = (e(64), torch.ones_like(wg), torch.ones_like(wu))
    dx, dwg, dwu = tq.glu_backward(e(40), e(64), wg, wu, g, u, out=out)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()


def test_outputs_past_2_31_elements():
    """Offsets into h, g, u and dh pass 32 bits."""
    say("glu train large")
    M, N, K = 150_100, 14336, 64
    x, (wg, wu) = ref.normal(3, (200, K)), _weights(5, N, K)
    xd = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    xd[-200:] = x.cuda()
    h, g, u = tq.glu_forward(xd, wg.cuda(), wu.cuda())
    wh, wgv, wuv, pre, eg, eu = ref.glu64(x.double(), wg.double(), wu.double(), "silu")
    ref.check(h[-200:], wh, pre, "h")
    ref.check(u[-200:], wuv, eu, "u")
    dh = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    tail = ref.normal(9, (200, N))
    dh[-200:] = tail.cuda()
    got = tq.glu_backward(dh, xd, wg.cuda(), wu.cuda(), g, u)
    torch.cuda.synchronize()
    want, e = ref.backward64(tail.double(), x.double(), wg.double(), wu.double(),
                             g[-200:].double().cpu(), u[-200:].double().cpu(), "silu")
    ref.check(got[0][-200:], want[0], e[0], "dx")
    ref.check(got[1], want[1], e[1], "dwg")
    assert not got[0][:1000].any()


def test_graph_replays():
    say("glu train graph")
    M, N, K = 200, 264, 192
    p = [t.cuda() for t in _backward_problem(61, M, N, K)]
    ws = torch.empty(max(16, tq.glu_backward_workspace(M, N, K)), dtype=torch.uint8, device="cuda")
    fout = tuple(torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    bout = tuple(torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (N, K), (N, K)))

    def step():
        tq.glu_forward(*p[1:4], out=fout)
        tq.glu_backward(p[0], *p[1:4], fout[1], fout[2], out=bout, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        p[1].copy_(ref.normal(100 + i, (M, K)))
        step()
        want = [t.clone() for t in fout + bout]
        for t in fout + bout:
            t.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(fout + bout, want):
            assert torch.equal(a, b)

"""The norm into 8-bit rows, the values it stands for and its gradients, against
their formulas in float64 (tests/i8_reference.py): codes and sums bit for bit,
the rest within bounds derived there."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

EPS = 1e-6
# rows of every layout: within a wave, 4 and 16 waves, two passes; odd ones
SIZES = [(1, 1), (3, 7), (5, 64), (2, 509), (1, 1024), (9, 1000), (4, 2048), (7, 2051), (3, 4096), (2, 5000),
         (1, 8192), (2, 14336), (3, 16381), (2, 16392), (1, 40003)]


# enough rows that dw is the sum of the blocks' parts, at every layout
SUMS = [(4200, 64), (2100, 1000), (1100, 2000), (1100, 3001), (1100, 5001), (1100, 9001), (1100, 17000)]


def _case(seed, M, K, xt, rt, wt):
    x = ref.normal(seed, (M, K), 1.0, r8.TYPES[xt])
    r = None if rt is None else ref.normal(seed + 1, (M, K), 3.0, r8.TYPES[rt])
    w = None if wt is None else (1 + ref.normal(seed + 2, (K,), 0.2, torch.float32)).to(r8.TYPES[wt])
    return x, r, w


def _check(x, r, w, eps=EPS):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    M, K = x.shape
    st = tq.new_status()
    q, s, y = tq.rms_norm_i8(d(x), d(w), d(r), eps, status=st)
    h, y2, rstd = tq.rms_norm_forward(d(x), d(w), d(r), eps, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    q6, s6, r6, y6 = r8.norm64(x, r, w, eps)
    assert torch.equal(y.cpu(), y6) and torch.equal(y2.cpu(), y6)
    if w is not None and w.dtype == torch.float32 and y6.dtype == torch.float32:
        # 127 t has 55 bits: fp64 decides, and may decide otherwise at a border
        t = 127 * y6.double() * w.double()
        f = t / (t.abs().amax(1) / 127)[:, None]
        near = ((f - f.floor()) - 0.5).abs() < 2.0 ** -40
        assert ((q.cpu() == q6) | near).all()
    else:
        assert torch.equal(q.cpu().double(), q6)
    r8.within(s, s6, r8.ROW * s6, "scales")
    r8.within(rstd, r6, r8.ROW * r6, "rstd")
    v = q6 * s6[:, None]
    r8.within(h, v, (r8.half_step(torch.bfloat16) + 2 * r8.ROW) * v.abs(), "h")


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("types", ["bf16 bf16 bf16", "bf16 None bf16", "fp32 bf16 None", "bf16 fp32 bf16",
                                   "fp32 None fp32", "fp32 fp32 bf16"])
def test_forward(M, K, types):
    say("rms_norm", M, K, types)
    _check(*_case(M + K, M, K, *[None if t == "None" else t for t in types.split()]))


def test_many_rows():
    _check(*_case(5, 3001, 320, "bf16", "bf16", "bf16"))


def test_borders():
    """Values whose quotient is exactly half way, or next to it, at every code:
    top 127 2^j makes 127 t / top = t 2^-j."""
    n = torch.arange(-127, 127, dtype=torch.float64) + 0.5
    for j in (0, 3, -20, 30, -90, 90):  # beyond 2^60 and below 2^-60: fp64
        t = torch.cat([n, torch.tensor([127.0, -127.0])]) * 2.0 ** j
        for step in (0, 1, -1):  # one unit of bf16 beside
            bits = t.to(torch.bfloat16).view(torch.int16) + step
            bits[-2:] -= step
            _check(bits.view(torch.bfloat16)[None, :].contiguous(), None, None)
    for seed in range(8):  # near borders: few bits in y, few in w
        x, _, w = _case(seed, 4, 4096, "bf16", None, "bf16")
        _check((x * 4).round() / 4, None, (w * 8).round() / 8)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -100, 2.0 ** 100, 2.0 ** 126])
@pytest.mark.parametrize("xt", ["bf16", "fp32"])
def test_far_from_one(scale, xt):
    x, _, w = _case(11, 3, 640, xt, None, "bf16")
    x = (x.double() * scale * 0.1).to(x.dtype)
    d = x.cuda()
    q, s, _ = tq.rms_norm_i8(d, w.cuda(), eps=1e-30)
    torch.cuda.synchronize()
    q6, s6, _, _ = r8.norm64(x, None, w, 1e-30)
    assert torch.equal(q.cpu().double(), q6)
    r8.within(s, s6, r8.ROW * s6 + 2.0 ** -149, "scales")


def test_zero_rows_and_rows_that_are_not_finite():
    for xt, K in (("bf16", 200), ("bf16", 3000), ("fp32", 200), ("bf16", 20000)):
        x, _, w = _case(3, 5, K, xt, None, "bf16")
        x[1] = 0
        x[2, K // 2] = float("inf")
        x[3, K - 1] = float("nan")
        st = tq.new_status()
        q, s, _ = tq.rms_norm_i8(x.cuda(), w.cuda(), status=st)
        h, _, _ = tq.rms_norm_forward(x.cuda(), w.cuda(), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == tq.DEV_NONFINITE
        keep = [0, 4]
        q6, s6, _, _ = r8.norm64(x[keep], None, w, EPS)
        assert torch.equal(q.cpu()[keep].double(), q6)
        r8.within(s.cpu()[keep], s6, r8.ROW * s6, "scales")
        assert (q.cpu()[1:4] == 0).all() and s.cpu()[1] == 0 and s.cpu()[2:4].isnan().all()
        assert (h.cpu()[1] == 0).all() and h.cpu()[2:4].isnan().all() and h.cpu()[keep].isfinite().all()


def test_sum_in_place_of_x():
    for K, t in ((333, "bf16"), (4096, "fp32"), (20000, "bf16")):
        x, r, w = _case(23, 6, K, t, t, "bf16")
        want = tq.rms_norm_i8(x.cuda(), w.cuda(), r.cuda())
        xd = x.cuda()
        q, s = torch.empty_like(want[0]), torch.empty_like(want[1])
        got = tq.rms_norm_i8(xd, w.cuda(), r.cuda(), out=(q, s, xd))
        torch.cuda.synchronize()
        assert got[2] is xd and all(torch.equal(a, b) for a, b in zip(got, want))


def test_sum_in_place_of_the_residual():
    for K in (333, 4096, 20000):
        x, r, w = _case(21, 6, K, "bf16", "bf16", "bf16")
        want = tq.rms_norm_i8(x.cuda(), w.cuda(), r.cuda())
        rd = r.cuda()
        q, s = torch.empty_like(want[0]), torch.empty_like(want[1])
        got = tq.rms_norm_i8(x.cuda(), w.cuda(), rd, out=(q, s, rd))
        torch.cuda.synchronize()
        assert got[2] is rd and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,K", SIZES + [(300, 513), (70, 17000)] + SUMS)
@pytest.mark.parametrize("types", ["bf16 bf16 1", "fp32 bf16 1", "bf16 fp32 0", "fp32 None 1", "bf16 None 0"])
def test_backward(M, K, types):
    yt, wt, add = types.split()
    say("rms_norm_backward", M, K, types)
    t = r8.TYPES[yt]
    y = ref.normal(31, (M, K), 2.0, t)
    w = None if wt == "None" else (1 + ref.normal(32, (K,), 0.2, torch.float32)).to(r8.TYPES[wt])
    dh = ref.normal(33, (M, K), 0.1)
    dy = ref.normal(34, (M, K), 0.1, t) if add == "1" else None
    rstd = (1 / (y.double().pow(2).mean(1) + EPS).sqrt()).float()
    d = lambda v: None if v is None else v.cuda()  # noqa: E731
    dx, dw = tq.rms_norm_backward(d(dh), d(y), d(rstd), d(w), d(dy))
    again, _ = tq.rms_norm_backward(d(dh), d(y), d(rstd), None if w is None else d(w), d(dy))
    torch.cuda.synchronize()
    (x6, xb), (w6, wb) = r8.norm_back64(dh, y, rstd, w, dy)
    r8.within(dx, x6, xb + r8.half_step(t) * x6.abs(), "dx")
    assert torch.equal(dx, again)
    if w is None:
        assert dw is None
    else:
        r8.within(dw, w6, wb + r8.half_step(w.dtype) * w6.abs(), "dw")


def test_gradient_against_differences():
    """RMSNorm's gradient is the norm's without the rounding: differences of
    sum(n w c) + sum(y e) in float64."""
    M, K = 3, 96
    x, r, w = _case(41, M, K, "fp32", "fp32", "fp32")
    c, e = ref.normal(44, (M, K), 1.0), ref.normal(45, (M, K), 1.0, torch.float32)
    xs = [t.cuda().requires_grad_() for t in (x, w, r)]
    h, y = tq.RMSNorm.apply(*xs)
    torch.autograd.backward([h, y], [c.cuda(), e.cuda()])

    def f(x, w, r):
        y = x + r
        return ((y / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt() * w) * c.double()).sum() + (y * e.double()).sum()

    step = 1e-6
    for i, t in enumerate(xs):
        at = [v.detach().cpu().double() for v in xs]
        direction = ref.normal(50 + i, tuple(t.shape), 1.0, torch.float32).double()
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * direction, at[i] - step * direction
        slope = float(f(*up) - f(*down)) / (2 * step)
        mine = float((t.grad.cpu().double() * direction).sum())
        size = float((t.grad.cpu().double() * direction).abs().sum())
        # the gradient's own bound (2^-17 of its terms), and the differences'
        # (third derivatives of order one: step^2; roundings of f over the step)
        assert abs(slope - mine) <= 2.0 ** -15 * size + 1e-8 * size, (i, slope, mine)


def test_autograd_parts():
    x, r, w = [t.cuda().requires_grad_() for t in _case(61, 5, 130, "fp32", "bf16", "bf16")]
    h, y = tq.RMSNorm.apply(x, w, r)
    assert h.dtype == torch.bfloat16 and y.dtype == torch.bfloat16
    g = torch.autograd.grad(y.float().sum(), (x, r), retain_graph=True)  # the sum alone
    assert (g[0] == 1).all() and (g[1] == 1).all() and g[0].dtype == torch.float32 and g[1].dtype == torch.bfloat16
    gx, gw, gr = torch.autograd.grad(h.float().square().sum(), (x, w, r))
    assert gx.dtype == torch.float32 and gw.dtype == torch.bfloat16 and torch.equal(gx, gr.float())
    h1 = tq.RMSNorm.apply(x.detach().to(torch.bfloat16), w)
    h1.sum().backward()
    assert isinstance(h1, torch.Tensor)
    (gg,) = torch.autograd.grad(tq.RMSNorm.apply(x, w).float().sum(), x, create_graph=True)
    with pytest.raises(tq.TQError, match="gradients of gradients"):
        gg.sum().backward()


def test_no_rows():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    q, s, y = tq.rms_norm_i8(x, w, x)
    assert q.shape == (0, 64) and s.shape == (0,) and y.shape == (0, 64)
    dx, dw = tq.rms_norm_backward(x, x, torch.empty(0, device="cuda"), w, out=(x, torch.full_like(w, 3)))
    torch.cuda.synchronize()
    assert (dw == 0).all()

"""tq_glu on the GPU against the float64 formula: h = act(x Wg^T) * (x Wu^T)
on packed ternary weights, at row counts from none to several tiles, rows of
one group, column counts that fill no tile, both group sizes."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _problem(seed, M, N, K, G, x=None):
    gate, up = ref.packed_weight(seed, N, K, G), ref.packed_weight(seed + 1, N, K, G)
    x = ref.normal(seed + 2, (M, K)) if x is None else x
    return x, gate, up


def _run(x, gate, up, N, K, G, act="silu", **kw):
    st = tq.new_status()
    h = tq.glu(x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up), N, K, G, act=act,
               status=st, **kw)
    torch.cuda.synchronize()
    return h, int(st.item())


def _check(x, gate, up, N, K, G, act, what):
    h, st = _run(x, gate, up, N, K, G, act)
    assert st == 0 and h.dtype == torch.bfloat16
    want, _, _, pre, _, _ = ref.glu64(x.double(), ref.weight64(*gate, N, K, G),
                                      ref.weight64(*up, N, K, G), act)
    ref.check(h, want, pre, what)
    return h


@pytest.mark.parametrize("G", [64, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 8, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 129, 200, 255, 257])
def test_rows(M, G):
    say("glu rows", M, G)
    N, K = 272, 640
    _check(*_problem(M, M, N, K, G), N, K, G, "silu" if M % 2 else "gelu", "M=%d" % M)


@pytest.mark.parametrize("M,N,K,G", [
    (1, 1, 64, 64), (1, 1, 128, 128), (5, 3, 128, 64), (4, 17, 192, 64), (16, 33, 384, 128),
    (1, 3584, 1024, 128), (7, 1000, 4096, 64), (20, 511, 2176, 128), (70, 129, 64, 64),
    (300, 1, 256, 128), (513, 257, 128, 128), (1, 96, 14336, 128), (3, 40, 14400, 64),
    (16, 64, 14336, 64), (64, 48, 7296, 128), (600, 700, 320, 64)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_shapes(M, N, K, G, act):
    say("glu shape", M, N, K, G, act)
    _check(*_problem(7, M, N, K, G), N, K, G, act, "M=%d N=%d K=%d G=%d" % (M, N, K, G))


@pytest.mark.parametrize("M,N,K,G", [(512, 3584, 1024, 128), (1029, 3600, 576, 64), (2048, 2049, 1152, 128)])
def test_prompts(M, N, K, G):
    say("glu prompt", M, N, K, G)
    _check(*_problem(11, M, N, K, G), N, K, G, "silu", "M=%d N=%d K=%d G=%d" % (M, N, K, G))


@pytest.mark.parametrize("M", [1, 12, 40, 300, 1100])
def test_magnitudes(M):
    """Rows of very large, very small, zero and widely spread values, and
    scales that are subnormal and near the top of fp16, keep the accuracy of
    an fp32 sum."""
    say("glu magnitudes", M)
    N, K, G = 2100 if M == 1100 else 144, 512, 128
    x, gate, up = _problem(23, M, N, K, G)
    f = x.float()
    for m in range(M):
        f[m] *= (1.0, 2.0 ** 40, 2.0 ** -60, 0.0, 2.0 ** -100, 1.0)[m % 6]
        if m % 6 == 5:
            f[m] *= torch.from_numpy(np.exp2(np.random.default_rng(m).integers(-30, 3, K)).astype(np.float32))
    x = f.to(torch.bfloat16)
    for i, (p, s) in enumerate((gate, up)):
        s[0::5] = 2.0 ** -24 * 3
        s[1::5] = 60000.0
        s[2::5] = -0.02                   # a stored scale may carry a sign
    for act in ("silu", "gelu"):
        wg, wu = ref.weight64(*gate, N, K, G), ref.weight64(*up, N, K, G)
        want, _, _, pre, _, _ = ref.glu64(x.double(), wg, wu, act)
        h, st = _run(x, gate, up, N, K, G, act)
        ok = want.abs() < 1e37            # where bf16 holds the result
        got = h.double().cpu()
        err = (got - want).abs()
        tol = pre + 2.0 ** -8 * want.abs() + 1e-37
        assert st == 0 and (err <= tol)[ok].all(), (M, act)


@pytest.mark.parametrize("M", [1, 9, 40, 300, 1100])
def test_nonfinite_rows_stay_in_their_rows(M):
    say("glu nonfinite", M)
    N, K, G = 2100 if M == 1100 else 100, 256, 64
    x, gate, up = _problem(29, M, N, K, G)
    clean = x.clone()
    bad = [m for m in range(M) if m % 7 == 3]
    for i, m in enumerate(bad):
        x[m, (17 * i) % K] = (float("inf"), float("-inf"), float("nan"))[i % 3]
    h, st = _run(x, gate, up, N, K, G)
    h0, _ = _run(clean, gate, up, N, K, G)
    keep = torch.ones(M, dtype=torch.bool)
    keep[bad] = False
    assert st == 0
    assert torch.equal(h.cpu()[keep].view(torch.int16), h0.cpu()[keep].view(torch.int16))
    for i, m in enumerate(bad):
        if i % 3 == 2:
            assert not torch.isfinite(h[m].float()).any()


@pytest.mark.parametrize("M", [1, 16, 50, 300, 1100])
def test_invalid_bytes_set_the_status(M):
    say("glu invalid bytes", M)
    N, K, G = 2100 if M == 1100 else 80, 256, 128
    x, gate, up = _problem(31, M, N, K, G)
    for which in (0, 1):
        p = (gate, up)[which][0].clone()
        p[N - 1, -2] = 243 + 12 * which
        pair = ((p, gate[1]), up) if which == 0 else (gate, (p, up[1]))
        _, st = _run(x, *pair, N, K, G)
        assert st == tq.DEV_INVALID_BYTE
    _, st = _run(x, gate, up, N, K, G)
    assert st == 0


@pytest.mark.parametrize("M,N", [(1, 50), (13, 50), (40, 50), (300, 50), (1100, 2100)])
def test_any_alignment_of_packed_bytes_and_narrow_alignment_of_h(M, N):
    say("glu alignment", M)
    K, G = 640, 64
    x, gate, up = _problem(37, M, N, K, G)
    want, _ = _run(x, gate, up, N, K, G)
    for off in (1, 2, 3, 5):
        pairs = []
        for p, s in (gate, up):
            buf = torch.zeros(p.numel() + 16, dtype=torch.uint8, device="cuda")
            v = buf[off:off + p.numel()].view(p.shape)
            v.copy_(p)
            sb = torch.zeros(s.numel() + 8, dtype=torch.float16, device="cuda")
            sv = sb[off:off + s.numel()].view(s.shape)
            sv.copy_(s)
            pairs.append((v, sv))
        hb = torch.full((M * N + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = hb[off:off + M * N].view(M, N)
        h = tq.glu(x.cuda(), *pairs, N, K, G, out=out)
        torch.cuda.synchronize()
        assert torch.equal(h, want)
        assert (hb[:off] == 7).all() and (hb[off + M * N:] == 7).all(), "written outside h"


@pytest.mark.parametrize("M,N", [(1, 512), (16, 513), (64, 200), (300, 200), (1100, 2100)])
def test_repeats_are_identical_on_any_stream_and_workspace(M, N):
    say("glu repeat", M, N)
    K, G = 1152, 128
    x, gate, up = _problem(41, M, N, K, G)
    want, _ = _run(x, gate, up, N, K, G)
    xd, gd, ud = x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up)
    need = tq.glu_workspace(M, N, K, G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.full((max(need, 16),), 0xA5, dtype=torch.uint8, device="cuda")
        got = [tq.glu(xd, gd, ud, N, K, G, workspace=ws) for _ in range(3)]
    side.synchronize()
    for h in got:
        assert torch.equal(h, want)


def test_no_rows():
    _, gate, up = _problem(43, 1, 48, 128, 64)
    h, st = _run(torch.zeros(0, 128, dtype=torch.bfloat16), gate, up, 48, 128, 64)
    assert h.shape == (0, 48) and st == 0


def test_more_than_2_31_outputs():
    """Offsets into h pass 32 bits: the last rows equal a small call's."""
    say("glu large")
    M, N, K, G = 150_100, 14340, 64, 64
    x, gate, up = _problem(47, 300, N, K, G)
    xd = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    xd[-300:] = x.cuda()
    h = tq.glu(xd, tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up), N, K, G)
    torch.cuda.synchronize()
    want, _, _, pre, _, _ = ref.glu64(x.double(), ref.weight64(*gate, N, K, G),
                                      ref.weight64(*up, N, K, G), "silu")
    ref.check(h[-300:], want, pre, "last rows")
    assert not h[:1000].any() and not h[75_000:75_300].any()


def test_graph_replays():
    """Captured once, replayed with new inputs and eager work between."""
    say("glu graph")
    K, G, N = 640, 128, 300
    for M in (1, 24, 300):
        x, gate, up = _problem(53, M, N, K, G)
        xd, gd, ud = x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up)
        ws = torch.empty(max(16, tq.glu_workspace(M, N, K, G)), dtype=torch.uint8, device="cuda")
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        tq.glu(xd, gd, ud, N, K, G, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tq.glu(xd, gd, ud, N, K, G, out=out, workspace=ws)
        for i in range(3):
            xd.copy_(ref.normal(100 + i, (M, K)))
            want = tq.glu(xd, gd, ud, N, K, G)
            out.fill_(3.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)

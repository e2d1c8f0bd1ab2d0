"""The packed products of many rows (wide_kernel) with group scales at the
edges of fp16, scales on 2 bytes and outputs on 2 or 4, captured in a graph;
and long sums of every kernel in root mean square."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import ffn_statistics as stat
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

GLU = [(2100, 2100, 128, 128), (1100, 4100, 64, 64), (4100, 257, 7296, 64)]
LORA = [(4100, 4100, 64, 64), (511, 4100, 7296, 64)]
LONG = [(300, 257, 33024, 128), (270, 700, 16448, 64), (7, 100, 33024, 64), (32, 96, 14336, 128), (1100, 257, 33024, 128)]


def _problem(seed, M, N, K, G, edges):
    x, gate, up = ref.normal(seed, (M, K)), ref.packed_weight(seed + 1, N, K, G), ref.packed_weight(seed + 2, N, K, G)
    if edges:
        for _, s in (gate, up):
            s[0::5] = 2.0 ** -24 * 3
            s[1::5] = 60000.0
            s[2::5] = -0.02
    return x, gate, up


def _glu64(x, gate, up, N, K, G, act):
    wg, wu = (ref.weight64(*w, N, K, G).cuda() for w in (gate, up))
    x = x.cuda().double()
    h, g, u, pre, _, _ = ref.glu64(x, wg, wu, act)
    dev = 1.13 * stat.of_product(x, wg) * u.abs() + g.abs() * stat.of_product(x, wu) + 2.0 ** -18 * h.abs()
    return h, pre, dev


def _shifted(t, by):
    """The same values, starting `by` elements after an aligned address."""
    buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
    return buf[by:by + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("M,N,K,G", GLU)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_edges(M, N, K, G, act):
    say("wide scales glu", M, N, K, G, act)
    x, gate, up = _problem(3, M, N, K, G, True)
    h = tq.glu(x.cuda(), *[(_shifted(p, 5), _shifted(s, 1)) for p, s in (gate, up)], N, K, G, act=act)
    want, pre, _ = _glu64(x, gate, up, N, K, G, act)
    ref.check(h, want.cpu(), pre.cpu() + 1e-37, "edges")


@pytest.mark.parametrize("M,N,K,G", LORA)
def test_lora_edges(M, N, K, G):
    say("wide scales lora", M, N, K, G)
    n, R = 3, 16
    x, w, _ = _problem(5, M, N, K, G, True)
    ids = torch.arange(M, dtype=torch.int32) % (n + 1) - 1
    a, b, scaling = ref.normal(7, (n, R, K), K ** -0.5), ref.normal(8, (n, N, R), 0.3), torch.tensor([1.0, -0.5, 2.0])
    out = torch.full((M * N + 8,), 7.0, device="cuda")
    d = [t.cuda() for t in (ids, a, b, scaling)]
    y = tq.lora_matmul(x.cuda(), _shifted(w[0], 3), _shifted(w[1], 3), *d, N, K, G, out=out[1:1 + M * N].view(M, N))
    want, bound = ref.lora64(x.cuda().double(), ref.weight64(*w, N, K, G).cuda(), ids,
                             *(t.cuda().double() for t in (a, b, scaling)))
    ref.check(y, want.cpu(), bound.cpu(), "edges", bf16=False)
    assert out[0] == 7 and (out[1 + M * N:] == 7).all(), "written outside y"


@pytest.mark.parametrize("M,N,K,G", [(2100, 2100, 128, 128), (4100, 257, 7296, 64)])
def test_graph_replays(M, N, K, G):
    say("wide graph", M, N, K, G)
    x, gate, up = _problem(11, M, N, K, G, False)
    xd, gd, ud = x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up)
    ws = torch.empty(tq.glu_workspace(M, N, K, G) + 16, dtype=torch.uint8, device="cuda")
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


@pytest.mark.parametrize("M,N,K,G", LONG + GLU)
def test_long_sums(M, N, K, G):
    say("long sums", M, N, K, G)
    x, gate, up = _problem(13, M, N, K, G, False)
    h = tq.glu(x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up), N, K, G)
    want, _, dev = _glu64(x, gate, up, N, K, G, "silu")
    stat.check_rms(h, want, dev, "glu", True)

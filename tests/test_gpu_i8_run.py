"""The norm into 8-bit rows, the products and the products by expert as they are
used together: a block step by step against float64, in training's values, on a
side stream, two at once, and captured in HIP graphs that are replayed with
other inputs (the device synchronised and eager work done between replays)."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8

pytestmark = pytest.mark.gpu

D, F, E, TOP, G = 512, 384, 4, 2, 128  # width, experts' width, experts, of each token


class Block:
    """y = x + residual; norm; experts up (relu2); norm; experts down; their sum
    over a token's experts into the stream; norm; a projection with bias."""

    def __init__(self, tokens):
        self.tokens = tokens
        make = lambda seed, n, k: [t.cuda() for t in ref.packed_weight(seed, n, k, G)]  # noqa: E731
        self.up, self.down, self.head = make(1, E * F, D), make(2, E * D, F), make(3, 700, D)
        self.w = [(1 + ref.normal(4 + i, (n,), 0.1, torch.float32)).to(torch.bfloat16).cuda()
                  for i, n in enumerate((D, F, D))]
        self.bias = ref.normal(8, (700,), 0.5, torch.float32).cuda()
        self.x, self.res = (torch.empty((tokens, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.rows = torch.empty(tokens * TOP, dtype=torch.int32, device="cuda")
        self.status = tq.new_status()

    def load(self, seed):
        self.x.copy_(ref.normal(seed, self.x.shape))
        self.res.copy_(ref.normal(seed + 1, self.x.shape, 2.0))
        rng = np.random.default_rng(seed)
        of = np.stack([rng.permutation(E)[:TOP] for _ in range(self.tokens)]).flatten()
        order = np.argsort(of, kind="stable")
        self.off.copy_(torch.from_numpy(np.searchsorted(of[order], np.arange(E + 1)).astype(np.int32)))
        self.rows.copy_(torch.from_numpy((order // TOP).astype(np.int32)))
        self.back = torch.from_numpy(np.argsort(order, kind="stable")).cuda().view(self.tokens, TOP)

    def run(self):
        st = self.status
        q, s, y = tq.rms_norm_i8(self.x, self.w[0], self.res, status=st)
        up = tq.expert_gemm_i8(q, s, *self.up, self.off, F, D, G, self.rows, act="relu2", status=st)
        q2, s2, _ = tq.rms_norm_i8(up, self.w[1], status=st)
        down = tq.expert_gemm_i8(q2, s2, *self.down, self.off, D, F, G, status=st)
        return q, s, y, up, q2, s2, down

    def end(self, y, down):
        both = down[self.back].float().sum(1).to(torch.bfloat16)
        q3, s3, y3 = tq.rms_norm_i8(both, self.w[2], y, status=self.status)
        return both, q3, s3, y3, tq.gemm_i8(q3, s3, *self.head, 700, D, G, self.bias, dtype=torch.float32,
                                            status=self.status)

    def check(self, q, s, y, up, q2, s2, down, both, q3, s3, y3, logits):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        c = lambda t: t.cpu()  # noqa: E731
        off, rows = c(self.off), c(self.rows).long()
        for (qq, ss, yy), (x, r, w) in (((q, s, y), (self.x, self.res, self.w[0])), ((q2, s2, up), (up, None, self.w[1])),
                                        ((q3, s3, y3), (both, y, self.w[2]))):
            q6, s6, _, y6 = r8.norm64(c(x), None if r is None else c(r), c(w), 1e-6)
            assert torch.equal(c(qq).double(), q6) and torch.equal(c(yy), y6)
            r8.within(ss, s6, r8.ROW * s6, "scales")
        for got, x, xs, (p, sc), n, k, act in ((up, c(q)[rows], c(s)[rows], self.up, F, D, "relu2"),
                                               (down, c(q2), c(s2), self.down, D, F, None)):
            p, sc = c(p).view(E, n, -1), c(sc).view(E, n, -1)
            for e in range(E):
                a, b = int(off[e]), int(off[e + 1])
                if a < b:
                    want, bound = r8.product64(x[a:b], xs[a:b], p[e], sc[e], n, k, G, act=act)
                    r8.within(got[a:b], want, bound, "expert %d" % e)
        want, bound = r8.product64(c(q3), c(s3), c(self.head[0]), c(self.head[1]), 700, D, G, c(self.bias),
                                   out=torch.float32)
        r8.within(logits, want, bound, "head")


@pytest.mark.parametrize("tokens", [1, 3, 17, 200])
def test_block(tokens):
    b = Block(tokens)
    for seed in (10, 20):
        b.load(seed)
        first = b.run()
        b.check(*first, *b.end(first[2], first[6]))


def test_training_sees_what_serving_computes():
    """rms_norm_forward's h times the dequantized weights, in float64, is
    gemm_i8's result to within h's rounding."""
    x, r = ref.normal(1, (9, D)).cuda(), ref.normal(2, (9, D), 2.0).cuda()
    w = (1 + ref.normal(3, (D,), 0.1, torch.float32)).to(torch.bfloat16).cuda()
    p, s = [t.cuda() for t in ref.packed_weight(4, 300, D, G)]
    q, qs, _ = tq.rms_norm_i8(x, w, r)
    h, _, _ = tq.rms_norm_forward(x, w, r)
    y = tq.gemm_i8(q, qs, p, s, 300, D, G, dtype=torch.float32)
    w6 = ref.weight64(p.cpu(), s.cpu(), 300, D, G)
    h6 = h.cpu().double()
    want = h6 @ w6.t()
    size = h6.abs() @ w6.abs().t()
    # h is q s to half a step of bf16 (2^-8 of q s, so 2^-8 (1 + 2^-7) of h), s to ROW, fp32 sums
    r8.within(y, want, (2.0 ** -8 * (1 + 2.0 ** -7) + 2 * r8.ROW + 2.0 ** -18) * size, "serving")


def test_side_stream_and_two_at_once():
    """Calls follow the current stream; two on two streams, each with its own
    workspace, give what they give one after the other."""
    shapes = [(700, 1024, 4992, 128), (650, 1024, 4992, 128)]  # with splits: workspaces
    data = []
    for i, (m, n, k, g) in enumerate(shapes):
        q, qs = r8.rows_i8(i, m, k)
        p, s = ref.packed_weight(i + 5, n, k, g)
        data.append([t.cuda() for t in (q, qs, p, s)])
        assert tq.gemm_i8_workspace(m, n, k, g) > 0
    want = [tq.gemm_i8(*d, n, k, g) for d, (m, n, k, g) in zip(data, shapes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[], []]
    for _ in range(5):
        for i, (st, d, (m, n, k, g)) in enumerate(zip(streams, data, shapes)):
            with torch.cuda.stream(st):
                x = torch.cat([d[0], d[0][:1]])[:m]  # made on this stream
                got[i].append(tq.gemm_i8(x, *d[1:], n, k, g))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("tokens", [2, 150])
def test_block_in_a_graph(tokens):
    b = Block(tokens)
    b.load(1)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.run()
    for seed in (3, 4, 5, 6):
        b.load(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = b.run()  # eager work between replays
        torch.cuda.synchronize()
        for i, (a, w) in enumerate(zip(out, want)):
            assert torch.equal(a, w), (seed, i)
        b.check(*out, *b.end(out[2], out[6]))


@pytest.mark.parametrize("M,N,K,G", [(778, 5000, 128, 128), (3099, 2600, 128, 128), (1350, 1024, 4992, 128),
                                     (6, 80, 14336, 64)])
def test_two_graphs_share_a_workspace(M, N, K, G):
    """A workspace that both calls are given, one after the other on a stream."""
    need = tq.gemm_i8_workspace(M, N, K, G)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    p, s = [t.cuda() for t in ref.packed_weight(2, N, K, G)]
    ins = [[t.cuda() for t in r8.rows_i8(i, M, K)] for i in range(2)]
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in ins]
    want = [tq.gemm_i8(*x, p, s, N, K, G) for x in ins]
    graphs = []
    for x, y in zip(ins, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tq.gemm_i8(*x, p, s, N, K, G, out=y, workspace=ws)
    for _ in range(3):
        ws.fill_(0xFF)
        for y in outs:
            y.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(outs, want))


@pytest.mark.parametrize("K", [512, 4096, 17000])
def test_training_in_a_graph(K):
    """Forward and backward captured (no eager graph of the same leaves lives
    then); every replay equals the eager call."""
    x = ref.normal(1, (70, K)).cuda().requires_grad_()
    r = ref.normal(2, (70, K), 2.0).cuda().requires_grad_()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda").requires_grad_()
    c = ref.normal(3, (70, K), 0.1).cuda()

    def step():
        h, y = tq.RMSNorm.apply(x, w, r)
        return torch.autograd.grad([h, y], [x, w, r], [c, c])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6, 7):
        with torch.no_grad():
            x.copy_(ref.normal(seed, (70, K)))
            c.copy_(ref.normal(seed + 10, (70, K), 0.1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed

"""8-bit rows times packed ternary weights, by themselves and grouped by expert,
against the formula in float64 within the bounds of tests/i8_reference.py."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

SHAPES = [(1, 64, 64), (16, 64, 64), (17, 128, 128), (33, 192, 64), (100, 320, 64), (48, 640, 128),
          (257, 1024, 128), (130, 1088, 64), (700, 3584, 128), (70, 14336, 64), (20, 14336, 128)]
ROWS = [1, 3, 4, 5, 8, 9, 16, 17, 32, 33, 65, 130, 260, 600]


def _inputs(seed, M, N, K, G, bias, res, out):
    q, qs = r8.rows_i8(seed, M, K)
    p, s = ref.packed_weight(seed + 1, N, K, G)
    b = None if bias is None else ref.normal(seed + 2, (N,), 0.5, r8.TYPES[bias])
    r = ref.normal(seed + 3, (M, N), 1.0, r8.TYPES[out]) if res else None
    return q, qs, p, s, b, r


def _d(t):
    return None if t is None else t.cuda()


def _check(seed, M, N, K, G, bias=None, act=None, res=False, out="bf16"):
    q, qs, p, s, b, r = _inputs(seed, M, N, K, G, bias, res, out)
    st = tq.new_status()
    y = tq.gemm_i8(q.cuda(), qs.cuda(), p.cuda(), s.cuda(), N, K, G, _d(b), act, _d(r), r8.TYPES[out], status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want, bound = r8.product64(q, qs, p, s, N, K, G, b, act, r, r8.TYPES[out])
    assert y.dtype == r8.TYPES[out] and y.shape == (M, N)
    r8.within(y, want, bound, "gemm_i8 %s" % ((M, N, K, G, bias, act, res, out),))


@pytest.mark.parametrize("N,K,G", SHAPES)
@pytest.mark.parametrize("M", ROWS)
def test_product(M, N, K, G):
    say("gemm_i8", M, N, K, G)
    _check(M + K, M, N, K, G, out="fp32")


@pytest.mark.parametrize("M", [2, 40, 270])
@pytest.mark.parametrize("bias,act,res,out", [
    ("bf16", None, False, "bf16"), ("fp32", "silu", True, "bf16"), (None, "gelu", False, "fp32"),
    ("bf16", "relu2", True, "fp32"), (None, None, True, "bf16"), (None, "relu2", False, "bf16")])
def test_epilogue(M, bias, act, res, out):
    for N in (64, 101):  # columns by fours, and one by one
        _check(7 * M, M, N, 768, 128, bias, act, res, out)


def test_one_hot_rows_are_exact():
    """A row with one code and scale 1 gives the weight itself."""
    for M, K, G in ((5, 320, 64), (130, 384, 128)):
        N = 37
        p, s = ref.packed_weight(3, N, K, G)
        w = ref.weight64(p, s, N, K, G)
        q = torch.zeros((M, K), dtype=torch.int8)
        at = np.random.default_rng(4).integers(0, K, M)
        q[torch.arange(M), torch.from_numpy(at)] = 1
        y = tq.gemm_i8(q.cuda(), torch.ones(M).cuda(), p.cuda(), s.cuda(), N, K, G, dtype=torch.float32)
        assert torch.equal(y.cpu().double(), w[:, torch.from_numpy(at)].t())
    # every place of a row at once
    for K, G in ((320, 64), (384, 128), (64, 64)):
        p, s = ref.packed_weight(5, N, K, G)
        q = torch.eye(K, dtype=torch.int8)
        y = tq.gemm_i8(q.cuda(), torch.ones(K).cuda(), p.cuda(), s.cuda(), N, K, G, dtype=torch.float32)
        assert torch.equal(y.cpu().double(), ref.weight64(p, s, N, K, G).t())


def _segments(rng, E, T, kind):
    if kind == "even":
        cuts = np.linspace(0, T, E + 1)
    elif kind == "one":
        cuts = np.where(np.arange(E + 1) > E // 2, T, 0)
    else:  # uneven, some empty, rows of none before and behind
        cuts = np.sort(rng.integers(T // 10, T - T // 10 + 1, E + 1))
    return cuts.astype(np.int32)


@pytest.mark.parametrize("T,E,N,K,G", [(1, 1, 16, 64, 64), (2, 5, 40, 128, 128), (16, 8, 130, 320, 64),
                                       (40, 3, 65, 1024, 128), (64, 70, 33, 192, 64), (300, 5, 257, 640, 128),
                                       (700, 3, 48, 704, 64), (900, 130, 20, 256, 128), (1100, 2, 300, 1024, 128)])
@pytest.mark.parametrize("kind", ["even", "one", "ragged"])
@pytest.mark.parametrize("gather", [False, True])
def test_experts(T, E, N, K, G, kind, gather):
    say("expert_gemm_i8", T, E, N, K, G, kind, gather)
    rng = np.random.default_rng(T + E)
    off = _segments(rng, E, T, kind)
    sources = max(1, T // 2) if gather else T
    q, qs = r8.rows_i8(T, sources, K)
    rows = torch.from_numpy(rng.integers(0, sources, T).astype(np.int32)) if gather else None
    p, s = ref.packed_weight(E, E * N, K, G)
    bias = ref.normal(9, (E, N), 0.5)
    res = ref.normal(10, (T, N), 1.0)
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    st = tq.new_status()
    tq.expert_gemm_i8(q.cuda(), qs.cuda(), p.cuda(), s.cuda(), torch.from_numpy(off).cuda(), N, K, G, _d(rows),
                      bias.cuda(), "relu2", res.cuda(), status=st, out=out)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    x, xs = (q, qs) if rows is None else (q[rows.long()], qs[rows.long()])
    nb = p.numel() // (E * N)
    left = torch.ones(T, dtype=torch.bool)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        left[a:b] = False
        if a < b:
            want, bound = r8.product64(x[a:b], xs[a:b], p.view(E, N, nb)[e], s.view(E, N, -1)[e], N, K, G, bias[e],
                                       "relu2", res[a:b])
            r8.within(out[a:b], want, bound, "expert %d" % e)
    assert (out.cpu()[left] == 7.0).all()


def test_many_rows_of_one_expert_among_many():
    """Far more rows than the mean: units of one segment by many blocks."""
    T, E, N, K, G = 200, 64, 50, 256, 128
    off = np.array([0] * 30 + [190] * 34 + [200], np.int32)
    q, qs = r8.rows_i8(1, T, K)
    p, s = ref.packed_weight(2, E * N, K, G)
    y = tq.expert_gemm_i8(q.cuda(), qs.cuda(), p.cuda(), s.cuda(), torch.from_numpy(off).cuda(), N, K, G,
                          dtype=torch.float32)
    nb = p.numel() // (E * N)
    for e in (29, 63):
        a, b = int(off[e]), int(off[e + 1])
        want, bound = r8.product64(q[a:b], qs[a:b], p.view(E, N, nb)[e], s.view(E, N, -1)[e], N, K, G,
                                   out=torch.float32)
        r8.within(y[a:b], want, bound, "expert %d" % e)

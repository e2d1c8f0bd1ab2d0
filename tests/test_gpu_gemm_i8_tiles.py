"""8-bit rows times packed ternary weights at sizes that reach every kernel:
samples of rows and columns, tiles' borders among them, against the formula in
float64 within the bounds of tests/i8_reference.py, and all results of rows that
pick one weight each against that weight."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

EPILOGUES = [("bf16", None, True, "bf16"), (None, "relu2", False, "bf16"), ("fp32", "gelu", True, "fp32"),
             ("fp32", "silu", False, "fp32")]


def _some(rng, n, most):
    """Up to about `most` of 0 .. n - 1: the ends, borders of 64 and 256, and others."""
    at = {0, n - 1, *(b + d for b in (64, 128, 256, n // 256 * 256) for d in (-1, 0)), *rng.integers(0, n, most)}
    return torch.tensor(sorted(i for i in at if 0 <= i < n))


def _run(q, qs, p, s, off, rows, N, K, G, bias, act, res, out, y, st):
    d = [None if t is None else t.cuda() for t in (q, qs, p, s, off, rows, bias, res)]
    if off is None:
        return tq.gemm_i8(d[0], d[1], d[2], d[3], N, K, G, d[6], act, d[7], out, st, y)
    return tq.expert_gemm_i8(d[0], d[1], d[2], d[3], d[4], N, K, G, d[5], d[6], act, d[7], out, st, y)


@pytest.mark.parametrize("case", range(len(r8.MIDDLE) + len(r8.LARGE)))
def test_samples(case):
    M, N, K, G, E = (r8.MIDDLE + r8.LARGE)[case]
    bt, act, with_res, ot = EPILOGUES[case % 4]
    say("gemm_i8 samples", M, N, K, G, E, bt, act, with_res, ot)
    rng = np.random.default_rng(case)
    off = torch.from_numpy(r8.segments(rng, E, M)) if E else None
    gather = E > 0 and case % 2 == 0
    sources = M // 2 + 1 if gather else M
    rows = torch.from_numpy(rng.integers(0, sources, M).astype(np.int32)) if gather else None
    q, qs = r8.rows_i8(case, sources, K)
    p, s = ref.packed_weight(case + 1, max(E, 1) * N, K, G)
    out = r8.TYPES[ot]
    bias = None if bt is None else ref.normal(case + 2, (max(E, 1), N) if E else (N,), 0.5, r8.TYPES[bt])
    res = ref.normal(case + 3, (M, N), 1.0, out) if with_res else None
    y = torch.full((M, N), 7.0, dtype=out, device="cuda")
    st = tq.new_status()
    _run(q, qs, p, s, off, rows, N, K, G, bias, act, res, out, y, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    y = y.cpu()
    x, xs = (q, qs) if rows is None else (q[rows.long()], qs[rows.long()])
    left = torch.ones(M, dtype=torch.bool)
    for e in range(max(E, 1)):
        a, b = (int(off[e]), int(off[e + 1])) if E else (0, M)
        if a == b:
            continue
        left[a:b] = False
        m, n = a + _some(rng, b - a, 40 if E > 1 else 120), _some(rng, N, 150)
        pe, se = p.view(max(E, 1), N, -1)[e][n], s.view(max(E, 1), N, -1)[e][n]
        be = None if bias is None else (bias[e] if E else bias)[n]
        want, bound = r8.product64(x[m], xs[m], pe, se, len(n), K, G, be, act,
                                   None if res is None else res[m][:, n], out)
        r8.within(y[m][:, n], want, bound, "expert %d" % e)
    assert (y[left] == 7.0).all()
    assert y.isfinite().all()


@pytest.mark.parametrize("M,N,K,G,E", [c for c in r8.LARGE if c[2] <= 4224])
def test_rows_that_pick_a_weight(M, N, K, G, E):
    """Rows with one code v at place k: v times the weight, exactly, everywhere."""
    say("gemm_i8 picks", M, N, K, G, E)
    rng = np.random.default_rng(K)
    at = torch.from_numpy(rng.integers(0, K, M))
    v = torch.from_numpy(rng.integers(-128, 128, M).astype(np.int8))
    q = torch.zeros((M, K), dtype=torch.int8)
    q[torch.arange(M), at] = v
    p, s = ref.packed_weight(K, N, K, G)
    off = None
    if E:  # every expert the same weights
        off = torch.from_numpy(r8.segments(rng, E, M))
        p, s = p.repeat(E, 1), s.repeat(E, 1)
    y = torch.zeros((M, N), dtype=torch.float32, device="cuda")
    _run(q, torch.ones(M), p, s, off, None, N, K, G, None, None, None, torch.float32, y, None)
    w = ref.weight64(p[:N], s[:N], N, K, G).float().cuda()
    want = w[:, at.cuda()].t() * v.cuda().float()[:, None]
    if E:
        want[:int(off[0])] = 0
        want[int(off[E]):] = 0
    assert torch.equal(y, want)

"""tq_lora_matmul for few rows and ranks, where one launch makes t and y (A of
up to 60 KB a block) and just past that: ranks, rows, both group sizes, one
and several splits of K, ids absent, out of range and repeated."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _run(x, w, ids, a, b, scaling, N, K, G, **kw):
    st = tq.new_status()
    y = tq.lora_matmul(*(t.cuda() for t in (x, *w, ids, a, b, scaling)), N, K, G, status=st, **kw)
    torch.cuda.synchronize()
    return y, int(st.item())


def _problem(seed, M, N, K, G, n, R):
    rng = np.random.default_rng(seed)
    return [ref.normal(seed, (M, K)), ref.packed_weight(seed + 1, N, K, G),
            torch.from_numpy(rng.integers(-1, n, M).astype(np.int32)),
            ref.normal(seed + 2, (n, R, K), K ** -0.5), ref.normal(seed + 3, (n, N, R), 0.3),
            ref.normal(seed + 4, (n,), 1.0, torch.float32)]


@pytest.mark.parametrize("M,N,K,G,R", [
    (1, 1, 128, 128, 8), (1, 33, 192, 64, 8), (1, 1024, 3584, 128, 8), (1, 50, 1024, 64, 32), (1, 50, 1088, 64, 32),
    (2, 77, 1984, 64, 8), (3, 500, 640, 128, 16), (5, 129, 384, 128, 16), (16, 240, 256, 64, 8), (16, 240, 128, 128, 16),
    (1, 16, 4096, 64, 8), (1, 16, 4224, 64, 8), (16, 100, 8192, 128, 8), (1, 40, 33024, 64, 8), (4, 60, 128, 64, 64),
    (1, 100, 128, 128, 256), (16, 31, 192, 64, 8)])
def test_formula(M, N, K, G, R):
    say("lora few", M, N, K, G, R)
    n = 3
    x, w, ids, a, b, scaling = _problem(M + R, M, N, K, G, n, R)
    ids[0] = 2
    y, st = _run(x, w, ids, a, b, scaling, N, K, G)
    want, bound = ref.lora64(x.double(), ref.weight64(*w, N, K, G), ids, a.double(), b.double(), scaling.double())
    assert st == 0
    ref.check(y, want, bound, "lora few %d %d %d" % (M, N, K), bf16=False)


@pytest.mark.parametrize("M,K", [(1, 1024), (4, 1024), (9, 384)])
def test_ids_and_named_adapters(M, K):
    say("lora few ids", M, K)
    N, G, n, R = 70, 64, 4, 8
    x, w, ids, a, b, scaling = _problem(50 + M, M, N, K, G, n, R)
    ids = torch.where(ids == 3, 1, ids).to(torch.int32)
    want, _ = _run(x, w, ids, a, b, scaling, N, K, G)
    a2, b2 = a.clone(), b.clone()
    a2[3], b2[3] = float("nan"), float("inf")
    ws = torch.full((max(16, tq.lora_workspace(M, N, K, G, R)),), 0xFF, dtype=torch.uint8, device="cuda")
    y, st = _run(x, w, ids, a2, b2, scaling, N, K, G, workspace=ws)
    assert st == 0 and torch.equal(y, want)
    if M > 2:
        x2 = x.clone()
        x2[2] = float("inf")
        y, _ = _run(x2, w, ids, a, b, scaling, N, K, G)
        keep = torch.arange(M) != 2
        assert torch.equal(y.cpu()[keep], want.cpu()[keep]) and not torch.isfinite(y[2]).any()
    for bad in (n, -2, 2 ** 31 - 1, -2 ** 31):
        wrong, none = ids.clone(), ids.clone()
        wrong[M - 1], none[M - 1] = bad, -1
        y, st = _run(x, w, wrong, a, b, scaling, N, K, G)
        y0, st0 = _run(x, w, none, a, b, scaling, N, K, G)
        assert st == tq.DEV_BAD_ADAPTER and st0 == 0 and torch.equal(y, y0)
    y, st = _run(x, w, torch.full((M,), -1, dtype=torch.int32), a[:0], b[:0], scaling[:0], N, K, G)
    y0, _ = _run(x, w, torch.full((M,), -1, dtype=torch.int32), a, b, scaling, N, K, G)
    assert st == 0 and torch.equal(y, y0)

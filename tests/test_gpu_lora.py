"""tq_lora_matmul on the GPU against the float64 formula: a packed ternary
projection beside each row's own low-rank adapter, with ids in any order,
absent, out of range, and adapters no row names."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _problem(seed, M, N, K, G, n, R):
    return {"x": ref.normal(seed, (M, K)), "w": ref.packed_weight(seed + 1, N, K, G),
            "a": ref.normal(seed + 2, (n, R, K), K ** -0.5), "b": ref.normal(seed + 3, (n, N, R), 0.3),
            "scaling": ref.normal(seed + 4, (n,), 1.0, torch.float32)}


def _ids(kind, M, n, seed=5):
    rng = np.random.default_rng(seed)
    if kind == "none":
        v = np.full(M, -1)
    elif kind == "mixed":
        v = rng.integers(-1, n, M)
    elif kind == "runs":
        v = np.sort(rng.integers(-1, n, M))
    else:
        v = np.full(M, n - 1)
    return torch.from_numpy(v.astype(np.int32))


def _run(p, ids, N, K, G, **kw):
    st = tq.new_status()
    y = tq.lora_matmul(p["x"].cuda(), p["w"][0].cuda(), p["w"][1].cuda(), ids.cuda(), p["a"].cuda(),
                       p["b"].cuda(), p["scaling"].cuda(), N, K, G, status=st, **kw)
    torch.cuda.synchronize()
    return y, int(st.item())


def _check(p, ids, N, K, G, what, status=0):
    y, st = _run(p, ids, N, K, G)
    assert st == status and y.dtype == torch.float32
    want, bound = ref.lora64(p["x"].double(), ref.weight64(*p["w"], N, K, G), ids, p["a"].double(),
                             p["b"].double(), p["scaling"].double())
    ref.check(y, want, bound, what, bf16=False)
    return y


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16, 17, 32, 33, 63, 64, 65, 128, 130, 257])
@pytest.mark.parametrize("kind", ["mixed", "runs", "none", "one"])
def test_rows_and_ids(M, kind):
    say("lora rows", M, kind)
    N, K, G = 208, 640, 64 if M % 2 else 128
    _check(_problem(M, M, N, K, G, 5, 16), _ids(kind, M, 5), N, K, G, "M=%d %s" % (M, kind))


@pytest.mark.parametrize("R", [8, 16, 24, 40, 64, 136, 256])
@pytest.mark.parametrize("M", [1, 20, 90, 300])
def test_ranks(R, M):
    say("lora rank", R, M)
    N, K, G = 147, 256, 128
    _check(_problem(R, M, N, K, G, 9, R), _ids("mixed", M, 9), N, K, G, "R=%d M=%d" % (R, M))


@pytest.mark.parametrize("M,N,K,G,n,R", [
    (1, 1, 64, 64, 1, 8), (3, 1, 128, 128, 2, 8), (1, 1024, 3584, 128, 4, 8),
    (32, 500, 14336, 128, 32, 16), (65, 33, 192, 64, 70, 24), (512, 2049, 1152, 128, 6, 64),
    (1030, 2048, 640, 64, 40, 16), (2048, 2064, 384, 128, 300, 32)])
def test_shapes(M, N, K, G, n, R):
    say("lora shape", M, N, K, G, n, R)
    for kind in ("mixed", "runs"):
        _check(_problem(7, M, N, K, G, n, R), _ids(kind, M, n), N, K, G, "M=%d N=%d %s" % (M, N, kind))


@pytest.mark.parametrize("M,N", [(1, 90), (19, 90), (80, 90), (400, 90), (1100, 2100)])
def test_bad_ids_are_flagged_and_count_as_none(M, N):
    say("lora bad ids", M)
    K, G, n = 256, 64, 3
    p = _problem(61, M, N, K, G, n, 16)
    ids = _ids("mixed", M, n)
    none = ids.clone()
    for m, v in ((0, n), (M // 2, -2), (M - 1, 2 ** 31 - 1)):
        ids[m], none[m] = v, -1
    y, st = _run(p, ids, N, K, G)
    want, st0 = _run(p, none, N, K, G)
    assert st == tq.DEV_BAD_ADAPTER and st0 == 0 and torch.equal(y, want)


@pytest.mark.parametrize("M,N", [(1, 90), (19, 90), (80, 90), (400, 90), (1100, 2100)])
def test_only_named_adapters_count(M, N):
    """NaN in adapters no row names, and in the rows of x of other requests,
    reaches nothing else; with no adapters the call is the projection alone."""
    say("lora named", M)
    K, G, n = 256, 128, 4
    p = _problem(67, M, N, K, G, n, 8)
    ids = torch.full((M,), -1, dtype=torch.int32)
    ids[::3] = 2
    want, _ = _run(p, ids, N, K, G)
    q = dict(p, a=p["a"].clone(), b=p["b"].clone(), scaling=p["scaling"].clone())
    for i in (0, 1, 3):
        q["a"][i] = float("nan")
        q["b"][i] = float("inf")
        q["scaling"][i] = float("nan")
    y, st = _run(q, ids, N, K, G)
    assert st == 0 and torch.equal(y, want)
    if M > 4:
        q["x"] = p["x"].clone()
        q["x"][3] = float("nan")
        y, _ = _run(q, ids, N, K, G)
        keep = torch.arange(M) != 3
        assert torch.equal(y.cpu()[keep], want.cpu()[keep]) and not torch.isfinite(y[3]).any()
    none = dict(p, a=p["a"][:0], b=p["b"][:0], scaling=p["scaling"][:0])
    y0, st = _run(none, torch.full((M,), -1, dtype=torch.int32), N, K, G)
    want0, bound0 = ref.lora64(p["x"].double(), ref.weight64(*p["w"], N, K, G), torch.full((M,), -1),
                               none["a"].double(), none["b"].double(), none["scaling"].double())
    assert st == 0
    ref.check(y0, want0, bound0, "no adapters", bf16=False)


@pytest.mark.parametrize("M,N", [(1, 512), (16, 513), (64, 200), (300, 200), (1100, 2100)])
def test_repeats_are_identical_on_any_stream_and_workspace(M, N):
    say("lora repeat", M, N)
    K, G, n, R = 1152, 128, 6, 16
    p = _problem(71, M, N, K, G, n, R)
    ids = _ids("mixed", M, n)
    want, _ = _run(p, ids, N, K, G)
    d = [t.cuda() for t in (p["x"], *p["w"], ids, p["a"], p["b"], p["scaling"])]
    need = tq.lora_workspace(M, N, K, G, R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN patterns
        got = [tq.lora_matmul(*d, N, K, G, workspace=ws) for _ in range(3)]
    side.synchronize()
    for y in got:
        assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 24, 300])
def test_graph_replays(M):
    say("lora graph", M)
    N, K, G, n, R = 300, 640, 64, 5, 16
    p = _problem(73, M, N, K, G, n, R)
    d = [t.cuda() for t in (p["x"], *p["w"], _ids("mixed", M, n), p["a"], p["b"], p["scaling"])]
    ws = torch.empty(max(16, tq.lora_workspace(M, N, K, G, R)), dtype=torch.uint8, device="cuda")
    out = torch.empty((M, N), dtype=torch.float32, device="cuda")
    tq.lora_matmul(*d, N, K, G, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.lora_matmul(*d, N, K, G, out=out, workspace=ws)
    for i in range(3):
        d[0].copy_(ref.normal(100 + i, (M, K)))
        d[3].copy_(_ids("mixed", M, n, seed=i))
        want = tq.lora_matmul(*d, N, K, G)
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_no_rows():
    p = _problem(79, 0, 48, 128, 64, 2, 8)
    y, st = _run(p, torch.zeros(0, dtype=torch.int32), 48, 128, 64)
    assert y.shape == (0, 48) and st == 0

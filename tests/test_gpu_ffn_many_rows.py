"""tq_glu and tq_lora_matmul at the sizes that take the 256 x 256 tiles or
split K between blocks: one and more rounds of tiles, K of one group, K longer
than a row's room in LDS, splits that do not divide it, tiles that N and M do
not fill.  Against the float64 formulas (computed on the GPU)."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

GLU = [  # tiles, one round or more, then K split: in 5 tiles' splits, 16, and 13 of 64-row chunks
    (1100, 4100, 64, 64), (8200, 513, 320, 64), (2100, 2100, 128, 128), (2048, 2049, 1152, 128),
    (4100, 257, 7296, 64), (1100, 257, 33024, 128), (270, 700, 16448, 64), (140, 520, 8192, 64)]
LORA = [
    (8200, 1029, 128, 128, 9, 24), (4100, 4100, 64, 64, 3, 8), (8200, 700, 2176, 128, 40, 64),
    (1500, 513, 17408, 128, 6, 40), (511, 4100, 7296, 64, 5, 16), (300, 1290, 16512, 128, 20, 72)]


def _glu_problem(seed, M, N, K, G):
    return ref.normal(seed, (M, K)), ref.packed_weight(seed + 1, N, K, G), ref.packed_weight(seed + 2, N, K, G)


def _glu(x, gate, up, N, K, G, act="silu", **kw):
    st = tq.new_status()
    h = tq.glu(x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up), N, K, G, act=act,
               status=st, **kw)
    torch.cuda.synchronize()
    return h, int(st.item())


def _lora_problem(seed, M, N, K, G, n, R):
    rng = np.random.default_rng(seed)
    return {"x": ref.normal(seed, (M, K)), "w": ref.packed_weight(seed + 1, N, K, G),
            "a": ref.normal(seed + 2, (n, R, K), K ** -0.5), "b": ref.normal(seed + 3, (n, N, R), 0.3),
            "scaling": ref.normal(seed + 4, (n,), 1.0, torch.float32),
            "ids": torch.from_numpy(rng.integers(-1, n, M).astype(np.int32))}


def _lora(p, N, K, G, **kw):
    st = tq.new_status()
    y = tq.lora_matmul(p["x"].cuda(), p["w"][0].cuda(), p["w"][1].cuda(), p["ids"].cuda(), p["a"].cuda(),
                       p["b"].cuda(), p["scaling"].cuda(), N, K, G, status=st, **kw)
    torch.cuda.synchronize()
    return y, int(st.item())


@pytest.mark.parametrize("M,N,K,G", GLU)
def test_glu(M, N, K, G):
    say("glu many rows", M, N, K, G)
    x, gate, up = _glu_problem(3, M, N, K, G)
    act = "gelu" if N % 2 else "silu"
    h, st = _glu(x, gate, up, N, K, G, act)
    wg, wu = (ref.weight64(*w, N, K, G).cuda() for w in (gate, up))
    want, _, _, pre, _, _ = ref.glu64(x.cuda().double(), wg, wu, act)
    assert st == 0
    ref.check(h, want.cpu(), pre.cpu(), "glu %d %d %d %d" % (M, N, K, G))


@pytest.mark.parametrize("M,N,K,G,n,R", LORA)
def test_lora(M, N, K, G, n, R):
    say("lora many rows", M, N, K, G, n, R)
    p = _lora_problem(5, M, N, K, G, n, R)
    y, st = _lora(p, N, K, G)
    want, bound = ref.lora64(p["x"].cuda().double(), ref.weight64(*p["w"], N, K, G).cuda(), p["ids"],
                             *(p[k].cuda().double() for k in ("a", "b", "scaling")))
    assert st == 0
    ref.check(y, want.cpu(), bound.cpu(), "lora %d %d %d %d" % (M, N, K, G), bf16=False)


@pytest.mark.parametrize("M,N,K,G", [(2100, 2100, 128, 128), (1100, 4100, 64, 64), (4100, 257, 7296, 64)])
def test_glu_rows_and_bytes(M, N, K, G):
    """Infinities and NaN stay in their rows; an invalid byte anywhere sets the
    status; packed bytes and h of any alignment; a workspace of NaN patterns;
    rows of very large and very small values."""
    say("glu many rows, rows and bytes", M, N, K, G)
    x, gate, up = _glu_problem(7, M, N, K, G)
    want, _ = _glu(x, gate, up, N, K, G)
    bad = torch.arange(3, M, 97)
    y = x.clone()
    for i, m in enumerate(bad.tolist()):
        y[m, (17 * i) % K] = (float("inf"), float("-inf"), float("nan"))[i % 3]
    h, st = _glu(y, gate, up, N, K, G)
    keep = torch.ones(M, dtype=torch.bool)
    keep[bad] = False
    assert st == 0 and torch.equal(h.cpu()[keep].view(torch.int16), want.cpu()[keep].view(torch.int16))
    assert not torch.isfinite(h[bad[2::3].cuda()].float()).any()

    for n, at in ((0, 0), (N - 1, -2), (N // 2, gate[0].shape[1] // 2)):
        q = up[0].clone()
        q[n, at] = 243
        assert _glu(x, gate, (q, up[1]), N, K, G)[1] == tq.DEV_INVALID_BYTE

    pairs = []
    for p, s in (gate, up):
        buf = torch.zeros(p.numel() + 16, dtype=torch.uint8, device="cuda")
        pairs.append((buf[3:3 + p.numel()].view(p.shape).copy_(p), s.cuda()))
    hb = torch.full((M * N + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((max(16, tq.glu_workspace(M, N, K, G)),), 0xFF, dtype=torch.uint8, device="cuda")
    out = tq.glu(x.cuda(), *pairs, N, K, G, out=hb[5:5 + M * N].view(M, N), workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert (hb[:5] == 7).all() and (hb[5 + M * N:] == 7).all(), "written outside h"

    scale = torch.tensor([1.0, 2.0 ** 30, 2.0 ** -60, 0.0])[torch.arange(M) % 4]
    z = (x.float() * scale[:, None]).to(torch.bfloat16)
    h, _ = _glu(z, gate, up, N, K, G)
    wg, wu = (ref.weight64(*w, N, K, G).cuda() for w in (gate, up))
    ref64, _, _, pre, _, _ = ref.glu64(z.cuda().double(), wg, wu, "silu")
    ref.check(h, ref64.cpu(), pre.cpu(), "glu magnitudes")


@pytest.mark.parametrize("M,N,K,G", [(2100, 4100, 128, 128), (8200, 700, 2176, 128)])
def test_lora_rows_and_adapters(M, N, K, G):
    """NaN in adapters that no row names and in other requests' rows reaches
    nothing else; ids out of range are flagged and count as none; repeats on a
    workspace of NaN patterns are identical."""
    say("lora many rows, rows and adapters", M, N, K, G)
    p = _lora_problem(11, M, N, K, G, 6, 16)
    p["ids"] = torch.where(p["ids"] == 4, 1, p["ids"]).to(torch.int32)   # nobody names 4
    want, st = _lora(p, N, K, G)
    assert st == 0
    q = dict(p, x=p["x"].clone(), a=p["a"].clone(), b=p["b"].clone())
    q["a"][4] = float("nan")
    q["b"][4] = float("inf")
    q["x"][259] = float("nan")
    ws = torch.full((max(16, tq.lora_workspace(M, N, K, G, 16)),), 0xFF, dtype=torch.uint8, device="cuda")
    y, st = _lora(q, N, K, G, workspace=ws)
    keep = torch.arange(M) != 259
    assert st == 0 and torch.equal(y.cpu()[keep], want.cpu()[keep]) and not torch.isfinite(y[259]).any()

    wrong, none = p["ids"].clone(), p["ids"].clone()
    for m, v in ((0, 6), (M // 2, -2), (M - 1, 2 ** 31 - 1)):
        wrong[m], none[m] = v, -1
    y, st = _lora(dict(p, ids=wrong), N, K, G)
    y0, st0 = _lora(dict(p, ids=none), N, K, G)
    assert st == tq.DEV_BAD_ADAPTER and st0 == 0 and torch.equal(y, y0)

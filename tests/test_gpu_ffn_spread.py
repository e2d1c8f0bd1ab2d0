"""tq_glu and tq_lora_matmul on rows whose elements spread over more than f16
holds: every sum as accurate as one in fp32, also where the row's largest
elements meet codes 0, cancel, or are infinitely far from the rest.

Tolerance: that of ffn_reference (K 2^-23 of the sum of magnitudes), which a
column that the largest elements do not reach takes from the others alone."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

# few_kernel in one and two tiles of rows, with one split and several; mid_kernel without and with splits, rows of
# one, two and four a block of the conversion; wide_kernel, one matrix and two, without and with splits, results
# stored by eights and singly; N and M that fill no tile
SHAPES = [(1, 64, 512, 128), (5, 100, 14336, 64), (16, 40, 192, 64), (20, 64, 512, 64), (32, 130, 4096, 128),
          (64, 96, 512, 128), (200, 260, 8192, 64), (300, 513, 17408, 128), (1100, 1030, 512, 128),
          (1100, 257, 7296, 64)]
WIDE_ONE = [(4100, 4100, 64, 64), (8200, 700, 2176, 128), (511, 4100, 7296, 64)]
WIDE_TWO = [(2100, 2104, 128, 128), (2048, 2049, 1152, 128), (4100, 257, 7296, 64)]


def _spread(kind, M, K, seed):
    """x in which small elements hide behind large ones that some columns do
    not see."""
    x = ref.normal(seed, (M, K)).float()
    at = K // 2 + 3
    if kind == "outlier":              # one element, growing from row to row
        x[:, at] = torch.exp2(torch.arange(M) % 90 + 20.0)
    elif kind == "lowest":             # the type's lowest value, as masks have it
        x[:, at] = -3.3895313892515355e38
        x[::2] *= 2.0 ** -20
    elif kind == "every scale":        # elements of every binade
        rng = np.random.default_rng(seed)
        x *= torch.from_numpy(np.exp2(rng.integers(-60, 60, (M, K))).astype(np.float32))
    else:                              # "tail": as an activation leaves them, 2^-15 .. 2^-100 beside ordinary ones
        g = 3 * x
        x = torch.where(g > 0, g, g * torch.exp2(8 * g))
    return x.to(torch.bfloat16)


def _weights(seed, N, K, G, at):
    """Half of the columns do not see element `at`."""
    w = ref.packed_weight(seed, N, K, G)
    p, B = w[0].view(N, K // G, -1), (G + 4) // 5
    byte, digit = at % G // 5, at % G % 5
    v = p[:, at // G, byte].to(torch.int32)
    v = v - (v // 3 ** digit % 3 - 1) * 3 ** digit
    p[::2, at // G, byte] = v[::2].to(torch.uint8)
    return p.view(N, -1), w[1]


@pytest.mark.parametrize("M,N,K,G", SHAPES + WIDE_ONE)
@pytest.mark.parametrize("kind", ["outlier", "lowest", "every scale", "tail"])
def test_projection_and_adapters(M, N, K, G, kind):
    say("lora spread", M, N, K, G, kind)
    x, w, n, R = _spread(kind, M, K, 3), _weights(5, N, K, G, K // 2 + 3), 3, 8
    rng = np.random.default_rng(9)
    ids = torch.from_numpy(rng.integers(-1, n, M).astype(np.int32))
    a, b = ref.normal(7, (n, R, K), K ** -0.5), ref.normal(8, (n, N, R), 0.3)
    a[:, :, K // 2 + 3] = 0
    scaling = torch.tensor([1.0, -0.5, 2.0])
    want, bound = ref.lora64(x.cuda().double(), ref.weight64(*w, N, K, G).cuda(), ids,
                             *(t.cuda().double() for t in (a, b, scaling)))
    ws = torch.full((tq.lora_workspace(M, N, K, G, R) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    args = [t.cuda() for t in (x, *w, ids, a, b, scaling)]
    y = tq.lora_matmul(*args, N, K, G, workspace=ws)
    again = tq.lora_matmul(*args, N, K, G)
    torch.cuda.synchronize()
    ref.check(y, want.cpu(), bound.cpu(), "lora %s" % kind, bf16=False)
    assert torch.equal(y, again)


@pytest.mark.parametrize("M,N,K,G", SHAPES + WIDE_TWO)
@pytest.mark.parametrize("kind", ["outlier", "every scale", "tail"])
def test_gated_block(M, N, K, G, kind):
    say("glu spread", M, N, K, G, kind)
    x, gate, up = _spread(kind, M, K, 11), _weights(13, N, K, G, K // 2 + 3), _weights(14, N, K, G, K // 2 + 3)
    act = "gelu" if M % 2 else "silu"
    wg, wu = (ref.weight64(*w, N, K, G).cuda() for w in (gate, up))
    want, _, _, pre, _, _ = ref.glu64(x.cuda().double(), wg, wu, act)
    args = [x.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up), N, K, G, act]
    ws = torch.full((tq.glu_workspace(M, N, K, G) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    h, again = tq.glu(*args, workspace=ws), tq.glu(*args)
    torch.cuda.synchronize()
    assert torch.equal(h.view(torch.int16), again.view(torch.int16))
    ok = (want.abs() < 1e37) & (pre < 1e37)          # where fp32 and bf16 hold the sums and the result
    zero = torch.zeros_like(want)
    ref.check(torch.where(ok, h.double(), zero).cpu(), torch.where(ok, want, zero).cpu(),
              torch.where(ok, pre, zero).cpu() + 1e-37, "glu %s" % kind)


@pytest.mark.parametrize("M", [3, 24, 70, 2100])
def test_nonfinite_rows_beside_spread_ones(M):
    """Rows with an infinity or NaN and a spread: nowhere finite, and nothing
    of theirs in the rows beside them."""
    say("spread nonfinite", M)
    N, K, G = (2104, 128, 128) if M == 2100 else (90, 512, 128)
    x, gate, up = _spread("outlier", M, K, 21), _weights(23, N, K, G, K // 2 + 3), _weights(24, N, K, G, K // 2 + 3)
    args = (tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up), N, K, G)
    want = tq.glu(x.cuda(), *args)
    bad = torch.arange(M) % 5 == 1
    x[bad, 7] = float("nan")
    h = tq.glu(x.cuda(), *args)
    torch.cuda.synchronize()
    assert not torch.isfinite(h[bad.cuda()].float()).any()
    assert torch.equal(h[~bad.cuda()].view(torch.int16), want[~bad.cuda()].view(torch.int16))

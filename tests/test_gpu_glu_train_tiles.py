"""tq_glu_forward and tq_glu_backward at the sizes that take 256 x 256 tiles,
several of them a block, both products side by side and one after the other, K
split and whole, against the float64 formulas (computed on the GPU): element by
element, and in root mean square against dg and du rounded as the call holds
them, so that nothing else is lost."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import ffn_statistics as stat
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

# what tests/test_ffn_plans.py says of them: the last number is N, padded to 64 or not, where dW is split
BACKWARD = [(4100, 3600, 1024, "silu"),   # side by side, dx split in 2
            (2048, 7168, 1024, "gelu"),   # side by side, 224 tiles of dW on 120 blocks, dx split in 4
            (2100, 3600, 1088, "silu"),   # one after the other, dx split in 4
            (4096, 1000, 576, "gelu"),    # dW split in 4, N padded
            (8200, 1000, 1024, "silu"),   # one after the other, dW split in 8
            (4500, 1024, 2048, "gelu")]   # neither split
FORWARD = [(4100, 3600, 1024, "silu"), (4100, 3601, 1024, "gelu"), (8200, 1000, 1024, "silu"), (3000, 3600, 512, "gelu")]


def _weights(seed, N, K):
    return ref.normal(seed, (N, K), 0.05).cuda(), ref.normal(seed + 1, (N, K), 0.05).cuda()


@pytest.mark.parametrize("M,N,K,act", FORWARD)
def test_forward(M, N, K, act):
    say("glu forward tiles", M, N, K, act)
    x, (wg, wu) = ref.normal(3, (M, K)).cuda(), _weights(5, N, K)
    got = tq.glu_forward(x, wg, wu, act)
    alone = tq.glu_forward(x, wg, wu, act, save=False)
    x, wg, wu = x.double(), wg.double(), wu.double()
    h, g, u, pre, eg, eu = ref.glu64(x, wg, wu, act)
    dg, du = stat.of_product(x, wg), stat.of_product(x, wu)
    for t, w, e, d, name in zip(got, (h, g, u), (pre, eg, eu),
                                (1.13 * dg * u.abs() + g.abs() * du + 2.0 ** -18 * h.abs(), dg, du), "hgu"):
        ref.check(t, w.cpu(), e.cpu(), name)
        stat.check_rms(t, w, d, name, True)
    assert torch.equal(alone, got[0])


@pytest.mark.parametrize("M,N,K,act", BACKWARD)
def test_backward(M, N, K, act):
    say("glu backward tiles", M, N, K, act)
    x, (wg, wu), dh = ref.normal(13, (M, K)).cuda(), _weights(15, N, K), ref.normal(17, (M, N)).cuda()
    g, u = ((x.double() @ w.double().t()).to(torch.bfloat16) for w in (wg, wu))
    args = (dh, x, wg, wu, g, u, act)
    ws = torch.full((tq.glu_backward_workspace(M, N, K) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    got = tq.glu_backward(*args, workspace=ws)          # a workspace of NaN patterns
    again = tq.glu_backward(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    d = [t.double() for t in args[:6]]
    want, pre = ref.backward64(*d, act)
    for t, w, e, name in zip(got, want, pre, ("dx", "dwg", "dwu")):
        ref.check(t, w.cpu(), e.cpu(), name)
    dg, du = stat.rounded_gates(d[0], d[4], d[5], ref.gate64(d[4], act))
    both, w = torch.cat([dg, du], 1), torch.cat([d[2], d[3]])
    for t, p, q, name in ((got[0], both, w.t().contiguous(), "dx"), (got[1], dg.t().contiguous(), d[1].t().contiguous(), "dwg"),
                          (got[2], du.t().contiguous(), d[1].t().contiguous(), "dwu")):
        # a gate within 2^-18 of the middle between two bf16 values may be rounded to the other one
        flips = 2.0 ** -8 * (2.0 ** -18 * 2 ** 9) ** 0.5 * (p.square() @ q.square().t()).sqrt()
        stat.check_rms(t, p @ q.t(), stat.of_product(p, q) + flips, name, True)

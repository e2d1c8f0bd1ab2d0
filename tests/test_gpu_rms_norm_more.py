"""The norm into 8-bit rows where tests/test_gpu_rms_norm.py does not look:
dweight from call to call, results that the C calls may leave out, and gradients
of some of the inputs alone."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.gpu_helpers import say
from tests.test_gpu_rms_norm import SIZES, SUMS

pytestmark = pytest.mark.gpu


def _inputs(M, K, yt, wt):
    y = ref.normal(31, (M, K), 2.0, r8.TYPES[yt])
    w = (1 + ref.normal(32, (K,), 0.2, torch.float32)).to(r8.TYPES[wt])
    dh, dy = ref.normal(33, (M, K), 0.1), ref.normal(34, (M, K), 0.1, r8.TYPES[yt])
    rstd = (1 / (y.double().pow(2).mean(1) + 1e-6).sqrt()).float()
    return [t.cuda() for t in (dh, y, rstd, w, dy)]


@pytest.mark.parametrize("M,K", SIZES + [(300, 513), (70, 17000), (1024, 3584), (1025, 3584), (2048, 1024)] + SUMS)
@pytest.mark.parametrize("types", ["bf16 bf16", "fp32 fp32"])
def test_gradients_repeat_bit_for_bit(M, K, types):
    """Both gradients, whatever the workspace holds: dweight is the sum of the
    blocks' parts, or made by blocks of columns."""
    say("rms_norm_backward again", M, K, types)
    dh, y, rstd, w, dy = _inputs(M, K, *types.split())
    need = tq.rms_norm_backward_workspace(M, K)
    first = None
    for fill in (0x00, 0xFF, 0x3C):
        ws = torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda")
        got = tq.rms_norm_backward(dh, y, rstd, w, dy, workspace=ws)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("M,K", [(5, 64), (300, 3584), (1100, 3001), (1100, 9001), (3, 17000)])
def test_results_that_may_be_left_out(M, K):
    """rstd of the forward call and dweight of the backward call may be NULL with
    a weight: the others are the same."""
    dh, y, rstd, w, dy = _inputs(M, K, "bf16", "bf16")
    lib, stream = tq.lib(), torch.cuda.current_stream().cuda_stream
    h, _, _ = tq.rms_norm_forward(y, w)
    h2 = torch.empty_like(h)
    assert lib.tq_rms_norm_forward(y.data_ptr(), 0, None, 0, w.data_ptr(), 0, M, K, 1e-6, h2.data_ptr(), None, None, None,
                                   stream) == 0
    dx, _ = tq.rms_norm_backward(dh, y, rstd, w, dy)
    dx2 = torch.empty_like(dx)
    need = tq.rms_norm_backward_workspace(M, K)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    assert lib.tq_rms_norm_backward(dh.data_ptr(), y.data_ptr(), 0, rstd.data_ptr(), w.data_ptr(), 0, dy.data_ptr(), M, K,
                                    dx2.data_ptr(), None, ws.data_ptr(), need, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(dx, dx2)


@pytest.mark.parametrize("which", [(0,), (1,), (2,), (0, 1), (1, 2), (0, 2)])
def test_gradients_of_some_inputs_alone(which):
    """Each input's gradient is what it is where all are asked for; the others
    get none."""
    t = [v.cuda() for v in (ref.normal(1, (7, 200)), (1 + ref.normal(2, (200,), 0.2, torch.float32)).to(torch.bfloat16),
                            ref.normal(3, (7, 200), 2.0))]
    c = ref.normal(4, (7, 200), 0.1).cuda()

    def grads(on):
        leaves = [v.clone().requires_grad_(i in on) for i, v in enumerate(t)]
        h, y = tq.RMSNorm.apply(*leaves)
        torch.autograd.backward([h, y], [c, c])
        return [v.grad for v in leaves]

    every, some = grads((0, 1, 2)), grads(which)
    for i in range(3):
        assert torch.equal(some[i], every[i]) if i in which else some[i] is None

"""eps of the norm into 8-bit rows: a row of zeros has rstd = eps^-1/2, which
gradients are multiplied by."""
import math

import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.test_i8_args import FWD, NORM, NULL, VALUE, _call

SMALLEST = math.ldexp(1.0, -252)


def test_an_eps_whose_root_leaves_fp32():
    """Refused where rstd is written, and only there."""
    for eps in (math.nextafter(SMALLEST, 0.0), 1e-80, 5e-324):
        assert _call("tq_rms_norm_forward", FWD, eps=eps) == VALUE
        assert _call("tq_rms_norm_forward", FWD, eps=eps, M=0) == VALUE
        assert _call("tq_rms_norm_forward", FWD, eps=eps, rstd=None, h=None) == NULL
        assert _call("tq_rms_norm_i8", NORM, eps=eps, q=None) == NULL
    assert _call("tq_rms_norm_forward", FWD, eps=SMALLEST, h=None) == NULL


@pytest.mark.gpu
@pytest.mark.parametrize("K,t", [(200, "bf16"), (3000, "fp32"), (17000, "bf16")])
def test_gradients_beside_a_row_of_zeros(K, t):
    """At the smallest eps a row of zeros adds nothing to dweight."""
    y = ref.normal(1, (4, K), 1.0, r8.TYPES[t])
    y[2] = 0
    w, dh = torch.ones(K), ref.normal(2, (4, K), 0.1)
    h, _, rstd = tq.rms_norm_forward(y.cuda(), w.cuda(), eps=SMALLEST)
    dx, dw = tq.rms_norm_backward(dh.cuda(), y.cuda(), rstd, w.cuda())
    with pytest.raises(tq.TQError):
        tq.rms_norm_forward(y.cuda(), w.cuda(), eps=1e-80)
    torch.cuda.synchronize()
    rstd = rstd.cpu()
    assert (h.cpu()[2] == 0).all() and rstd[2] == math.ldexp(1.0, 126)
    (x6, xb), (w6, wb) = r8.norm_back64(dh, y, rstd, w, None)
    r8.within(dx, x6, xb + r8.half_step(dx.dtype) * x6.abs(), "dx")
    r8.within(dw, w6, wb + r8.half_step(dw.dtype) * w6.abs(), "dw")

"""Calls of the norm into 8-bit rows and of its products on tensors of a device
that is not the current one enqueue with that device current and on its stream
(host tensors that say they are on device 1; nothing is launched)."""
import torch

import ternary_weight_only_amd as tq
from tests.test_devices import calls, one  # noqa: F401

M, N, K, G, E = 4, 8, 128, 64, 3


def _weights(n):
    from tests import ffn_reference as ref
    from tests.test_devices import OnOne
    p, s = ref.packed_weight(1, n, K, G)
    return p.as_subclass(OnOne), s.as_subclass(OnOne)


def test_calls(calls):  # noqa: F811
    x, w, r = one(M, K), one(K), one(M, K)
    q, s = one(M, K, dtype=torch.int8), one(M, dtype=torch.float32)
    h, rstd, y = one(M, K), one(M, dtype=torch.float32), one(M, N)
    ws = one(1 << 20, dtype=torch.uint8)
    off = one(E + 1, dtype=torch.int32)
    tq.rms_norm_i8(x, w, r, out=(q, s, r))
    tq.rms_norm_forward(x, w, r, out=(h, r, rstd))
    tq.rms_norm_backward(h, x, rstd, w, out=(x, w), workspace=ws)
    tq.gemm_i8(q, s, *_weights(N), N, K, G, out=y, workspace=ws)
    tq.expert_gemm_i8(q, s, *_weights(E * N), off, N, K, G, out=y, workspace=ws)
    assert calls == [(f, 1, 101) for f in ("tq_rms_norm_i8", "tq_rms_norm_forward", "tq_rms_norm_backward",
                                           "tq_gemm_i8", "tq_expert_gemm_i8")]

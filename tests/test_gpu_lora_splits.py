"""tq_lora_matmul where K is split between blocks and rows name many adapters
or few, in every kernel: the adapters' part by itself (scales 0), so that one
added twice or not at all cannot hide beside the projection, then with it.
Element by element, and in root mean square against what fp32 sums leave."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import ffn_statistics as stat
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

# M, N, K, G, adapters, ranks
MANY = [(64, 513, 14336, 128, 40, 16), (200, 520, 8192, 64, 40, 8), (300, 200, 16512, 128, 30, 8)]   # a result's own
FEW = [(64, 513, 14336, 128, 4, 16), (300, 1290, 16512, 128, 20, 72), (200, 300, 8192, 64, 2, 40)]   # one after another
WIDE = [(1500, 513, 17408, 128, 6, 40), (511, 4100, 7296, 64, 90, 16), (8200, 700, 2176, 128, 40, 64)]
LITTLE = [(24, 200, 4096, 64, 6, 16), (32, 500, 14336, 128, 32, 16), (17, 300, 16384, 64, 3, 200), (9, 200, 8192, 128, 5, 64),
          (1, 400, 14336, 128, 2, 8)]


@pytest.mark.parametrize("M,N,K,G,n,R", MANY + FEW + WIDE + LITTLE)
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_adapters_alone_and_beside_the_projection(M, N, K, G, n, R, order):
    say("lora splits", M, N, K, G, n, R, order)
    rng = np.random.default_rng(M + R)
    ids = rng.integers(-1, n, M)
    ids = torch.from_numpy((np.sort(ids) if order == "runs" else ids).astype(np.int32))
    x, (packed, scales) = ref.normal(3, (M, K)), ref.packed_weight(5, N, K, G)
    a, b = ref.normal(7, (n, R, K), K ** -0.5), ref.normal(8, (n, N, R), 0.3)
    scaling = ref.normal(9, (n,), 1.0, torch.float32)
    w64 = ref.weight64(packed, scales, N, K, G).cuda()
    x64, a64, b64, s64 = (t.cuda().double() for t in (x, a, b, scaling))
    part = stat.of_adapters(x64, ids, a64, b64, s64)
    for sc, w in ((torch.zeros_like(scales), torch.zeros_like(w64)), (scales, w64)):
        ws = torch.full((tq.lora_workspace(M, N, K, G, R) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        y = tq.lora_matmul(*(t.cuda() for t in (x, packed, sc, ids, a, b, scaling)), N, K, G, workspace=ws)
        want, bound = ref.lora64(x64, w, ids, a64, b64, s64)
        ref.check(y, want.cpu(), bound.cpu(), "scales %s" % bool(sc.any()), bf16=False)
        deviation = (part.square() + stat.of_product(x64, w).square()).sqrt()
        stat.check_rms(y, want, deviation, "scales %s" % bool(sc.any()), False)

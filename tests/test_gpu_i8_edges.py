"""Products of 8-bit rows at the narrowest results and in a padded batch, as
their documentation allows: one to seven columns, rows that no expert has
(before, behind and in a tile with others'), and the same row many times over."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 2, 7])
@pytest.mark.parametrize("M", [1, 9, 17, 40, 300])
@pytest.mark.parametrize("K,G", [(64, 64), (128, 64), (1984, 64), (128, 128), (1920, 128)])
def test_narrow_results(M, N, K, G):
    say("gemm_i8 narrow", M, N, K, G)
    q, qs = r8.rows_i8(M, M, K)
    p, s = ref.packed_weight(N, N, K, G)
    bias, res = ref.normal(3, (N,), 0.5), ref.normal(4, (M, N), 1.0)
    d = [t.cuda() for t in (q, qs, p, s)]
    y = res.cuda()
    tq.gemm_i8(*d, N, K, G, bias.cuda(), "silu", y, out=y)
    want, bound = r8.product64(q, qs, p, s, N, K, G, bias, "silu", res)
    r8.within(y, want, bound, "narrow")


@pytest.mark.parametrize("T,used,E,N,K,G", [(32, 9, 4, 130, 1024, 128), (32, 9, 4, 130, 1024, 64), (64, 3, 70, 33, 192, 64),
                                            (400, 150, 3, 260, 2176, 128), (400, 150, 3, 260, 2176, 64),
                                            (3000, 2500, 4, 2600, 256, 128), (3000, 2500, 4, 2600, 192, 64)])
def test_a_padded_batch(T, used, E, N, K, G):
    """Rows behind the last segment hold anything, row indices out of range too:
    none is read, none is written, and no status bit is set."""
    rng = np.random.default_rng(T)
    off = np.sort(rng.integers(0, used + 1, E + 1)).astype(np.int32)
    off[0], off[-1] = 0, used
    sources = max(1, used // 3)
    q, qs = r8.rows_i8(T, sources, K)
    p, s = ref.packed_weight(E, E * N, K, G)
    rows = torch.full((T,), -5, dtype=torch.int32)
    rows[:used] = torch.from_numpy(rng.integers(0, sources, used).astype(np.int32))
    rows[:min(used, 7)] = 0  # one row for many
    res = ref.normal(5, (T, N), 1.0)
    res[used:] = float("nan")
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    st = tq.new_status()
    tq.expert_gemm_i8(q.cuda(), qs.cuda(), p.cuda(), s.cuda(), torch.from_numpy(off).cuda(), N, K, G, rows.cuda(), None,
                      "relu2", res.cuda(), status=st, out=out)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (out[used:] == 7.0).all()
    nb = p.numel() // (E * N)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            at = rows[a:b].long()
            want, bound = r8.product64(q[at], qs[at], p.view(E, N, nb)[e], s.view(E, N, -1)[e], N, K, G, None, "relu2",
                                       res[a:b])
            r8.within(out[a:b], want, bound, "expert %d" % e)

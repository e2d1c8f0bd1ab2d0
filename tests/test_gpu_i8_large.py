"""The norm into 8-bit rows and its products past 32 bits of elements and bytes,
and at the longest rows."""
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def test_norm_of_more_than_32_bits_of_elements():
    """Rows do not depend on their number: 1056 copies of 1000 rows, 4.3e9
    elements, are the rows by themselves."""
    base, K, times = 1000, 4096, 1056
    x = ref.normal(1, (base, K)).cuda()
    w = (1 + ref.normal(2, (K,), 0.2, torch.float32)).to(torch.bfloat16).cuda()
    q1, s1, _ = tq.rms_norm_i8(x, w)
    h1, _, r1 = tq.rms_norm_forward(x, w)
    many = x.repeat(times, 1)
    assert many.numel() > 1 << 32
    q, s, _ = tq.rms_norm_i8(many, w)
    for i in (0, times // 2, times - 1):
        assert torch.equal(q[i * base:(i + 1) * base], q1) and torch.equal(s[i * base:(i + 1) * base], s1)
    del q
    h, _, r = tq.rms_norm_forward(many, w)
    for i in (0, times // 2, times - 1):
        assert torch.equal(h[i * base:(i + 1) * base], h1) and torch.equal(r[i * base:(i + 1) * base], r1)
    # gradients, with h as its own gradient: rows as by themselves, dw the sum
    dx1, dw1 = tq.rms_norm_backward(h1, x, r1, w)
    dx, dw = tq.rms_norm_backward(h, many, r, w)
    # the two may run different kernels: sums of a row differ by 2^-18 of their terms, then a rounding
    for i in (0, times // 2, times - 1):
        part = dx[i * base:(i + 1) * base].double()
        assert ((part - dx1.double()).abs() <= 2.0 ** -7 * dx1.double().abs() + 2.0 ** -12).all()
    n = x.double() * r1.double()[:, None]
    want, size = times * (h1.double() * n).sum(0), times * (h1.double() * n).abs().sum(0)
    # 256 blocks of 4125 rows each in a row, then ten additions
    assert ((dw.double() - want).abs() <= 4200 * 2.0 ** -24 * size + 2.0 ** -8 * want.abs()).all()


def test_results_of_more_than_32_bits_of_elements():
    M, N, K, G = 530000, 8200, 64, 64
    base = 1000
    q1, qs1 = [t.cuda() for t in r8.rows_i8(1, base, K)]
    p, s = [t.cuda() for t in ref.packed_weight(2, N, K, G)]
    q, qs = q1.repeat(M // base, 1), qs1.repeat(M // base)
    y1 = tq.gemm_i8(q1, qs1, p, s, N, K, G)
    y = tq.gemm_i8(q, qs, p, s, N, K, G)
    assert y.numel() > 1 << 32
    want, bound = r8.product64(q1[:64].cpu(), qs1[:64].cpu(), p.cpu(), s.cpu(), N, K, G)
    r8.within(y1[:64], want, bound, "alone")
    for i in (0, M // base // 2, M // base - 1):  # (one group: no order of sums to differ by)
        assert torch.equal(y[i * base:(i + 1) * base], y1)


@pytest.mark.parametrize("T", [12, 3700])
@pytest.mark.parametrize("G", [64, 128])
def test_weights_of_more_than_32_bits_of_bytes(T, G):
    """Experts at both ends and in the middle of 4.4e9 packed bytes."""
    N, K = 4096, 14336
    B = (G + 4) // 5
    E = (1 << 32) // (N * K // G * B) + 12
    say("experts", T, G, E)
    used = [0, E // 2, E - 1]
    p = torch.full((E, N, K // G * B), 121, dtype=torch.uint8, device="cuda")  # zeros
    s = torch.ones((E, N, K // G), dtype=torch.float16, device="cuda")
    for e in used:
        pe, se = ref.packed_weight(e, 64, K, G)
        p[e, -64:], s[e, -64:] = pe.cuda(), se.cuda()
    assert p.numel() > 1 << 32
    q, qs = r8.rows_i8(T, T, K)
    off = torch.zeros(E + 1, dtype=torch.int32)
    cut = [T // 3, T // 2, T]
    for e, c in zip(used, cut):
        off[e + 1:] = c
    st = tq.new_status()
    y = tq.expert_gemm_i8(q.cuda(), qs.cuda(), p, s, off.cuda(), N, K, G, dtype=torch.float32, status=st)
    assert int(st.item()) == 0
    for e, a, b in zip(used, [0] + cut, cut):
        rows = sorted({a, b - 1, (a + b) // 2})
        want, bound = r8.product64(q[rows], qs[rows], p[e, -64:].cpu(), s[e, -64:].cpu(), 64, K, G, out=torch.float32)
        r8.within(y[rows, -64:], want, bound, "expert %d" % e)
        assert (y[a:b, :-64] == 0).all()


@pytest.mark.parametrize("M,N,K,G", [(3, 20, 1 << 21, 128), (3, 20, (1 << 21) - 64, 64), (20, 40, 1 << 20, 64),
                                     (20, 40, (1 << 20) + 128, 128)])
def test_longest_rows(M, N, K, G):
    q, qs = r8.rows_i8(M, M, K)
    p, s = ref.packed_weight(N, N, K, G)
    y = tq.gemm_i8(q.cuda(), qs.cuda(), p.cuda(), s.cuda(), N, K, G, dtype=torch.float32)
    want, bound = r8.product64(q, qs, p, s, N, K, G, out=torch.float32)
    r8.within(y, want, bound, "K = %d" % K)
    # that bound is of all roundings in one direction; as they come, those of n = 2^14 partial
    # sums make about n 2^-24.5 of a term, 2^-17 of the root of the terms' squares
    x = q.double().view(M, K // G, G)
    parts = torch.einsum("mgj,ngj->mng", x, ref.weight64(p, s, N, K, G).view(N, K // G, G)) * qs.double()[:, None, None]
    assert ((y.cpu().double() - want).abs() <= 2.0 ** -12 * parts.square().sum(-1).sqrt() + 2.0 ** -20 * want.abs()).all()


@pytest.mark.parametrize("T,N,G", [(9, 100, 64), (300, 200, 64), (300, 200, 128), (3100, 2600, 128)])
def test_rows_given_by_index_of_32_bits_of_bytes(T, N, G):
    """Row indices up to the last of 2^32 bytes of x, one row more refused."""
    K, sources = 4096, 1 << 20
    x = torch.zeros((sources + 1, K), dtype=torch.int8, device="cuda")
    xs = torch.zeros(sources + 1, device="cuda")
    rows = torch.cat([torch.tensor([0, sources - 1, sources // 2, sources // 2 - 1]),
                      torch.randint(0, sources, (T - 4,), generator=torch.Generator().manual_seed(T))])
    q, qs = r8.rows_i8(T, T, K)
    _, first = torch.unique(rows, return_inverse=True)
    q, qs = q[first], qs[first]  # the same row for the same index
    x[rows.cuda()], xs[rows.cuda()] = q.cuda(), qs.cuda()
    p, s = [t.cuda() for t in ref.packed_weight(3, N, K, G)]
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    index = rows.int().cuda()
    y = tq.expert_gemm_i8(x[:sources], xs[:sources], p, s, off, N, K, G, index, dtype=torch.float32)
    some = list(range(4)) + list(range(4, T, max(1, T // 40)))
    want, bound = r8.product64(q[some], qs[some], p.cpu(), s.cpu(), N, K, G, out=torch.float32)
    r8.within(y[some], want, bound, "rows by index")
    with pytest.raises(tq.TQError):
        tq.expert_gemm_i8(x, xs, p, s, off, N, K, G, index, dtype=torch.float32)

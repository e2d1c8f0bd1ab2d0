"""The norm into 8-bit rows and the products that read them: what the binding
refuses before any launch, what the status word says, and values and addresses
at the edge (infinities, unaligned results, the residual in place, no rows)."""
import numpy as np
import pytest
import torch

import ternary_weight_only_amd as tq
from tests import ffn_reference as ref
from tests import i8_reference as r8

pytestmark = pytest.mark.gpu

M, N, K, G, E = 6, 48, 128, 64, 3


def _refused(call):
    with pytest.raises(tq.TQError):
        call()


def _product(M=M, N=N, K=K, G=G, E=0, seed=1):
    q, qs = r8.rows_i8(seed, M, K)
    p, s = ref.packed_weight(seed + 1, max(E, 1) * N, K, G)
    return [t.cuda() for t in (q, qs, p, s)]


def test_norm_refusals():
    x = ref.normal(1, (M, K)).cuda()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    for bad in (x.half(), x[:, ::2], x[0], x.cpu(), x.t(), None, 3):
        for call in (tq.rms_norm_i8, tq.rms_norm_forward):
            _refused(lambda: call(bad, w))
            if bad is not None:
                _refused(lambda: call(x, w, bad))
    for bad in (w[:-1], w.half(), w.cpu(), w[None]):
        _refused(lambda: tq.rms_norm_i8(x, bad))
    for eps in (0.0, -1.0, float("nan"), float("inf"), "1"):
        _refused(lambda: tq.rms_norm_i8(x, w, eps=eps))
    q = torch.full((M, K), 5, dtype=torch.int8, device="cuda")
    s, y = torch.full((M,), 5.0, device="cuda"), torch.full_like(x, 5.0)
    for out in ((q[:-1], s, None), (q, s.double(), None), (q.cpu(), s, None), (q, s, y), (q.float(), s, None)):
        _refused(lambda: tq.rms_norm_i8(x, w, out=out))
    _refused(lambda: tq.rms_norm_i8(x, w, x, out=(q, s, y.float())))
    _refused(lambda: tq.rms_norm_forward(x, w, out=(y.float(), None, s)))
    h, _, rstd = tq.rms_norm_forward(x, w)
    for bad in (h.float(), h[:-1], h.cpu(), h.t()):
        _refused(lambda: tq.rms_norm_backward(bad, x, rstd, w))
    for bad in (rstd[:-1], rstd.double(), rstd.cpu()):
        _refused(lambda: tq.rms_norm_backward(h, x, bad, w))
    _refused(lambda: tq.rms_norm_backward(h, x, rstd, w, x.float()))
    _refused(lambda: tq.rms_norm_backward(h, x, rstd, None, out=(None, w)))
    _refused(lambda: tq.rms_norm_backward(h, x, rstd, w, out=(y.float(), None)))
    _refused(lambda: tq.rms_norm_backward(h, x, rstd, w, workspace=torch.zeros(8, device="cuda")))
    torch.cuda.synchronize()
    assert (q == 5).all() and (s == 5).all() and (y == 5).all()


def test_product_refusals():
    q, qs, p, s = _product()
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    good = dict(x=q, x_scales=qs, packed=p, scales=s, N=N, K=K, G=G, out=out)

    def call(**kw):
        return tq.gemm_i8(**{**good, **kw})

    bias = torch.zeros(N, device="cuda")
    for kw in (dict(x=q.float()), dict(x=q[:, :64]), dict(x=q.t()), dict(x=q.cpu()), dict(x=q[0]), dict(x=None),
               dict(x_scales=qs[:-1]), dict(x_scales=qs.double()), dict(x_scales=qs.cpu()), dict(packed=p.flatten()[:-1]),
               dict(packed=p.to(torch.int8)), dict(scales=s.float()), dict(scales=s.cpu()), dict(G=32), dict(K=100),
               dict(N=N + 1), dict(bias=bias.half()), dict(bias=bias[:-1]), dict(bias=bias.cpu()), dict(act="tanh"),
               dict(act=2), dict(residual=out.float()), dict(residual=out[:-1]), dict(residual=out.t()),
               dict(dtype=torch.float16), dict(dtype=torch.float32), dict(out=out[:, :8]),
               dict(status=torch.zeros(1, device="cuda"))):
        _refused(lambda: call(**kw))
    q, qs, p, s = _product(E=E)
    off = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    rows = torch.zeros(M, dtype=torch.int32, device="cuda")
    given = dict(x=q, x_scales=qs, packed=p, scales=s, offsets=off, N=N, K=K, G=G, rows=rows, out=out)

    def experts(**kw):
        return tq.expert_gemm_i8(**{**given, **kw})

    for kw in (dict(offsets=off[:-1]), dict(offsets=off.long()), dict(offsets=off.cpu()), dict(offsets=off[:1]),
               dict(offsets=[0, 2, 2, 6]), dict(rows=rows.long()), dict(rows=rows[:-1]), dict(rows=rows[None]),
               dict(rows=rows.cpu()), dict(packed=p[:N]), dict(scales=s[:N]), dict(bias=bias),
               dict(bias=torch.zeros(E, N - 1, device="cuda")), dict(x=q[:, :64]), dict(out=out[:-1])):
        _refused(lambda: experts(**kw))
    torch.cuda.synchronize()
    assert (out == 3.0).all()
    # off the required alignment: the library's own check
    buf = torch.zeros(M * K + 16, dtype=torch.int8, device="cuda")
    _refused(lambda: call(x=buf[8:8 + M * K].view(M, K)))


# few rows, small tiles, splits, the large tile of each group size
STATUS = [(4, 48, 128, 128, 0), (5, 32, 14336, 64, 0), (40, 140, 1088, 64, 0), (65, 130, 2176, 128, 0),
          (778, 5000, 128, 128, 0), (3113, 2600, 64, 64, 0), (3099, 2600, 128, 128, 0)]


@pytest.mark.parametrize("M,N,K,G,_", STATUS)
def test_invalid_bytes(M, N, K, G, _):
    """One byte beyond 242 anywhere sets the bit, and no other row is touched."""
    q, qs, p, s = _product(M, N, K, G)
    st = tq.new_status()
    want = tq.gemm_i8(q, qs, p, s, N, K, G, status=st)
    assert int(st.item()) == 0
    rng = np.random.default_rng(M)
    for byte in (243, 255):
        n, b = int(rng.integers(N)), int(rng.integers(p.shape[1]))
        bad = p.clone()
        bad[n, b] = byte
        st.zero_()
        got = tq.gemm_i8(q, qs, bad, s, N, K, G, status=st)
        assert int(st.item()) == tq.DEV_INVALID_BYTE, (n, b, byte)
        keep = torch.arange(N, device="cuda") != n
        assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("T,N,K,G,E", [(20, 48, 320, 64, 9), (30, 64, 14336, 128, 6), (70, 90, 640, 128, 3),
                                       (60, 48, 2176, 64, 2), (976, 2600, 384, 128, 20), (2628, 2600, 128, 128, 20)])
def test_offsets_and_rows_out_of_range(T, N, K, G, E):
    q, qs, p, s = _product(T, N, K, G, E)
    off = torch.from_numpy(r8.segments(np.random.default_rng(T), E, T)).cuda()
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    st = tq.new_status()
    clean = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    tq.expert_gemm_i8(q, qs, p, s, off, N, K, G, rows, status=st, out=clean)
    assert int(st.item()) == 0
    # rows of no source count as zeros, others are as they were
    at = int(off[0])
    for bad in (-1, T, 2 ** 31 - 1, -2 ** 31):
        r = rows.clone()
        r[at] = bad
        y = torch.zeros_like(clean)
        st.zero_()
        tq.expert_gemm_i8(q, qs, p, s, off, N, K, G, r, status=st, out=y)
        assert int(st.item()) == tq.DEV_BAD_ROW
        assert (y[at] == 0).all()
        y[at] = clean[at]
        assert torch.equal(y, clean)
    for change in ((0, -5), (E, T + 1), (E, 2 ** 31 - 1), (E // 2, 2 ** 31 - 1), (E // 2, -2 ** 31), (0, T)):
        bad = off.clone()
        bad[change[0]] = change[1]
        st.zero_()
        tq.expert_gemm_i8(q, qs, p, s, bad, N, K, G, rows, status=st, out=torch.zeros_like(clean))
        assert int(st.item()) & tq.DEV_BAD_SEGMENT, change
    # a row index out of range in a row of no expert is never read
    if at > 0:
        r = rows.clone()
        r[0] = -7
        st.zero_()
        tq.expert_gemm_i8(q, qs, p, s, off, N, K, G, r, status=st, out=torch.zeros_like(clean))
        assert int(st.item()) == 0


@pytest.mark.parametrize("M,N,K,G,_", STATUS[:5])
def test_infinities_and_nan_stay_where_they_are(M, N, K, G, _):
    """Row scales, group scales, bias and residual that are not finite reach the
    results that use them and no others, through every activation."""
    q, qs, p, s = _product(M, N, K, G)
    inf, nan = float("inf"), float("nan")
    for act in (None, "relu2", "silu", "gelu"):
        bias, res = torch.zeros(N, device="cuda"), torch.zeros((M, N), device="cuda")
        args = dict(N=N, K=K, G=G, act=act, dtype=torch.float32)
        want = tq.gemm_i8(q, qs, p, s, bias=bias, residual=res, **args)
        b, r, x, sc = bias.clone(), res.clone(), qs.clone(), s.clone()
        b[3], b[7], r[1, 2], x[M - 1], sc[11, K // G - 1] = nan, inf, -inf, nan, nan
        got = tq.gemm_i8(q, x, p, sc, bias=b, residual=r, **args)
        hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
        hit[:, [3, 7, 11]] = True
        hit[M - 1] = True
        assert got[:, 3].isnan().all() and got[:, 11].isnan().all() and got[M - 1].isnan().all()
        assert (got[:M - 1, 7] == inf).all() and got[1, 2] == -inf
        hit[1, 2] = True
        assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("M,N,K,G,_", STATUS)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_addresses(M, N, K, G, _, out):
    """Results and residuals off 16 bytes, and the residual in place of the
    result, give the same results bit for bit; the memory around stays."""
    q, qs, p, s = _product(M, N, K, G)
    t = r8.TYPES[out]
    res = ref.normal(9, (M, N), 1.0, t).cuda()
    want = tq.gemm_i8(q, qs, p, s, N, K, G, residual=res, dtype=t)
    r = res.clone()
    assert tq.gemm_i8(q, qs, p, s, N, K, G, residual=r, dtype=t, out=r) is r
    assert torch.equal(r, want)
    buf = torch.full((M * N + 2,), 3.0, dtype=t, device="cuda")
    r1 = torch.cat([res.flatten()[:1], res.flatten()])[1:].view(M, N)  # one element on
    tq.gemm_i8(q, qs, p, s, N, K, G, residual=r1, dtype=t, out=buf[1:-1].view(M, N))
    assert torch.equal(buf[1:-1].view(M, N), want) and buf[0] == 3 and buf[-1] == 3
    # the packed bytes at any alignment
    for k in (1, 2, 3):
        moved = torch.zeros(p.numel() + k, dtype=torch.uint8, device="cuda")
        moved[k:] = p.flatten()
        assert torch.equal(tq.gemm_i8(q, qs, moved[k:].view(p.shape), s, N, K, G, residual=res, dtype=t), want)


def test_no_rows_and_no_rows_of_an_expert():
    q, qs, p, s = _product(E=E)
    empty = q[:0]
    y = tq.gemm_i8(empty, qs[:0], p[:N], s[:N], N, K, G)
    assert y.shape == (0, N)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    assert tq.expert_gemm_i8(empty, qs[:0], p, s, off, N, K, G).shape == (0, N)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert tq.expert_gemm_i8(empty, qs[:0], p, s, off, N, K, G, rows=none).shape == (0, N)
    for T, N2, K2, G2 in ((6, N, K, G), (100, 90, 2176, 128), (2628, 2600, 128, 128)):  # all segments empty
        q, qs, p, s = _product(T, N2, K2, G2, E)
        out = torch.full((T, N2), 4.0, dtype=torch.bfloat16, device="cuda")
        for at in (0, T // 2, T):
            off.fill_(at)
            st = tq.new_status()
            tq.expert_gemm_i8(q, qs, p, s, off, N2, K2, G2, status=st, out=out)
            assert int(st.item()) == 0 and (out == 4.0).all()
    with pytest.raises(tq.TQError):  # rows, but nothing that they could name
        tq.expert_gemm_i8(empty, qs[:0], p, s, off, N2, K2, G2, rows=torch.zeros(3, dtype=torch.int32, device="cuda"))


def test_the_same_row_for_every_expert():
    """Row indices may repeat: one token for all experts."""
    q, qs, p, s = _product(1, 80, 256, 128, 4)
    off = torch.arange(5, dtype=torch.int32, device="cuda")
    y = tq.expert_gemm_i8(q, qs, p, s, off, 80, 256, 128, rows=torch.zeros(4, dtype=torch.int32, device="cuda"),
                          dtype=torch.float32)
    for e in range(4):
        one = tq.gemm_i8(q, qs, p.view(4, 80, -1)[e], s.view(4, 80, -1)[e], 80, 256, 128, dtype=torch.float32)
        want, bound = r8.product64(q.cpu(), qs.cpu(), p.cpu().view(4, 80, -1)[e], s.cpu().view(4, 80, -1)[e], 80, 256, 128,
                                   out=torch.float32)
        r8.within(y[e:e + 1], want, bound, "expert %d" % e)
        r8.within(one, want, bound, "alone %d" % e)

"""The norm into 8-bit rows and the products that read them refuse bad arguments
on the host, before any HIP call.  No test here launches a kernel."""
import math
import os

import pytest

FAKE = 0x100000  # never dereferenced: every call below fails validation first


def _lib():
    import ternary_weight_only_amd as tq
    if not os.path.exists(tq.binding.LIB_PATH):
        from ternary_weight_only_amd import build
        build.build_library()
    return tq.lib()


NULL, SHAPE, GROUP, ALIGN, WORKSPACE, ACT, TYPE, VALUE = -1, -2, -3, -4, -6, -7, -8, -9
BIG = 1 << 40


def _call(fn, spec, **changed):
    """Call fn with the arguments of `spec` (name -> value), some changed."""
    assert not set(changed) - set(spec)
    return getattr(_lib(), fn)(*{**spec, **changed}.values())


NORM = dict(x=FAKE, xt=0, r=FAKE, rt=0, w=FAKE, wt=0, M=30, K=100, eps=1e-6, q=FAKE, s=FAKE, y=FAKE, st=None,
            stream=None)
FWD = dict(x=FAKE, xt=0, r=FAKE, rt=1, w=FAKE, wt=0, M=30, K=100, eps=1e-6, h=FAKE, y=FAKE, rstd=FAKE, st=None,
           stream=None)
BWD = dict(dh=FAKE, y=FAKE, yt=0, rstd=FAKE, w=FAKE, wt=1, dy=FAKE, M=30, K=100, dx=FAKE, dw=FAKE, ws=FAKE, wn=BIG,
           stream=None)
GEMM = dict(x=FAKE, xs=FAKE, p=FAKE, s=FAKE, b=FAKE, bt=0, act=2, r=FAKE, M=300, N=50, K=256, G=64, out=FAKE, ot=0,
            ws=FAKE, wn=BIG, st=None, stream=None)
EXPERT = dict(x=FAKE, xs=FAKE, sources=300, rows=FAKE, p=FAKE, s=FAKE, off=FAKE, E=4, b=FAKE, bt=0, act=2, r=FAKE,
              T=300, N=50, K=256, G=64, out=FAKE, ot=0, ws=FAKE, wn=BIG, st=None, stream=None)


@pytest.mark.parametrize("fn,spec,pointers", [
    ("tq_rms_norm_i8", NORM, ["x", "q", "s", "y", "r"]),
    ("tq_rms_norm_forward", FWD, ["x", "h", "y", "r"]),
    ("tq_rms_norm_backward", BWD, ["dh", "y", "rstd", "dx", "w"]),
    ("tq_gemm_i8", GEMM, ["x", "xs", "p", "s", "out"]),
    ("tq_expert_gemm_i8", EXPERT, ["x", "xs", "p", "s", "off", "out"])])
def test_null_pointers(fn, spec, pointers):
    for p in pointers:
        assert _call(fn, spec, **{p: None}) == NULL, p


def test_shapes():
    for fn, spec in (("tq_rms_norm_i8", NORM), ("tq_rms_norm_forward", FWD), ("tq_rms_norm_backward", BWD)):
        for bad in (dict(M=-1), dict(K=0), dict(K=-3), dict(K=(1 << 21) + 1), dict(M=(1 << 30) + 1),
                    dict(M=1 << 30, K=2048)):
            assert _call(fn, spec, **bad) == SHAPE, (fn, bad)
    for fn, spec, m in (("tq_gemm_i8", GEMM, "M"), ("tq_expert_gemm_i8", EXPERT, "T")):
        for bad in ({m: -1}, dict(N=0), dict(K=0), dict(K=100), dict(K=(1 << 21) + 64), {m: 1 << 31},
                    dict(N=1 << 31), dict(N=1 << 30, K=4096), dict(K=192, G=128)):
            assert _call(fn, spec, **bad) == SHAPE, (fn, bad)
        for G in (0, 32, 96, 256, -64):
            assert _call(fn, spec, G=G) == GROUP
    for bad in (dict(E=0), dict(E=-1), dict(E=65537), dict(E=65536, N=1 << 20), dict(sources=-1),
                dict(sources=0), dict(rows=None, sources=299), dict(sources=(1 << 24) + 1)):
        assert _call("tq_expert_gemm_i8", EXPERT, **bad) == SHAPE, bad


def test_rows_by_index_reach_32_bits():
    """Offsets into x have 32 bits where rows are given, and only there."""
    assert _call("tq_expert_gemm_i8", EXPERT, sources=(1 << 24) + 1, rows=FAKE) == SHAPE
    assert _call("tq_expert_gemm_i8", EXPERT, sources=1 << 24, x=None) == NULL
    assert _call("tq_expert_gemm_i8", EXPERT, sources=(1 << 24) + 1, rows=None, x=None) == NULL


def test_types_and_numbers():
    for fn, spec, types in (("tq_rms_norm_i8", NORM, ["xt", "rt", "wt"]), ("tq_rms_norm_forward", FWD, ["xt", "rt", "wt"]),
                            ("tq_rms_norm_backward", BWD, ["yt", "wt"]), ("tq_gemm_i8", GEMM, ["bt", "ot"]),
                            ("tq_expert_gemm_i8", EXPERT, ["bt", "ot"])):
        for t in types:
            for bad in (-1, 2, 99):
                assert _call(fn, spec, **{t: bad}) == TYPE, (fn, t)
    for fn, spec in (("tq_rms_norm_i8", NORM), ("tq_rms_norm_forward", FWD)):
        for eps in (0.0, -1e-6, math.inf, math.nan):
            assert _call(fn, spec, eps=eps) == VALUE
    for fn, spec in (("tq_gemm_i8", GEMM), ("tq_expert_gemm_i8", EXPERT)):
        for act in (-1, 4, 99):
            assert _call(fn, spec, act=act) == ACT


def test_alignment():
    for fn, spec, by2, by4, by16 in (
            ("tq_rms_norm_i8", NORM, ["x", "r", "y", "w"], ["s", "st"], []),
            ("tq_rms_norm_forward", FWD, ["x", "h", "w"], ["r", "y", "rstd", "st"], []),
            ("tq_rms_norm_backward", {**BWD, "M": 30000}, ["dh", "y", "dy", "dx"], ["rstd", "w", "dw"], ["ws"]),
            ("tq_gemm_i8", GEMM, ["s", "b", "r", "out"], ["xs", "st"], ["x"]),
            ("tq_expert_gemm_i8", EXPERT, ["s", "b", "r", "out"], ["xs", "st", "rows", "off"], ["x"])):
        for names, off in ((by2, 1), (by4, 2), (by16, 8)):
            for n in names:
                assert _call(fn, spec, **{n: FAKE + off}) == ALIGN, (fn, n)


def test_workspaces():
    lib = _lib()
    need = lib.tq_rms_norm_backward_workspace(30000, 100)
    assert need > 0 and lib.tq_rms_norm_backward_workspace(30, 100) == 0
    assert _call("tq_rms_norm_backward", BWD, M=30000, wn=need - 1) == WORKSPACE
    assert _call("tq_rms_norm_backward", BWD, M=30000, ws=None) == NULL
    shapes = [(M, N, K, G) for M in (1, 5, 20, 33, 100, 300, 5000) for N, K in ((50, 256), (1024, 14336), (9000, 8192))
              for G in (64, 128)]
    some = 0
    for M, N, K, G in shapes:
        need = lib.tq_gemm_i8_workspace(M, N, K, G)
        assert need >= 0
        if need:
            some += 1
            args = dict(M=M, N=N, K=K, G=G)
            assert _call("tq_gemm_i8", GEMM, wn=need - 1, **args) == WORKSPACE
            assert _call("tq_gemm_i8", GEMM, ws=None, **args) == NULL
            assert _call("tq_gemm_i8", GEMM, ws=FAKE + 8, **args) == ALIGN
    assert some
    assert lib.tq_gemm_i8_workspace(-1, 50, 256, 64) == 0 and lib.tq_gemm_i8_workspace(30, 50, 100, 64) == 0
    assert lib.tq_expert_gemm_i8_workspace(30, 50, 256, 64, 0) == 0
    assert lib.tq_rms_norm_backward_workspace(0, 64) == 0 and lib.tq_rms_norm_backward_workspace(4, 0) == 0


def test_nothing_to_do():
    assert _call("tq_rms_norm_i8", NORM, M=0, x=None, q=None) == 0
    assert _call("tq_rms_norm_forward", FWD, M=0, h=None) == 0
    assert _call("tq_gemm_i8", GEMM, M=0, x=None, out=None) == 0
    assert _call("tq_expert_gemm_i8", EXPERT, T=0, x=None, off=None, sources=0) == 0


def test_status_strings():
    lib = _lib()
    names = [lib.tq_status_string(rc).decode() for rc in (TYPE, VALUE)]
    assert "TQ_ERR_TYPE" in names[0] and "TQ_ERR_VALUE" in names[1]

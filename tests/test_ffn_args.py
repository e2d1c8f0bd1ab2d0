"""The gated feed-forward and adapter calls refuse bad arguments on the host,
before any HIP call.  No test here launches a kernel."""
import os

import pytest
import torch

FAKE = 0x100000  # never dereferenced: every call below fails validation first


def _lib():
    import ternary_weight_only_amd as tq
    if not os.path.exists(tq.binding.LIB_PATH):
        from ternary_weight_only_amd import build
        build.build_library()
    return tq.lib()


NULL, SHAPE, GROUP, ALIGN, WORKSPACE, ACT = -1, -2, -3, -4, -6, -7
BIG = 1 << 40


def _call(fn, spec, **changed):
    """Call fn with the arguments of `spec` (name -> value), some changed."""
    assert not set(changed) - set(spec)
    return getattr(_lib(), fn)(*{**spec, **changed}.values())


GLU = dict(x=FAKE, gp=FAKE, gs=FAKE, up=FAKE, us=FAKE, M=300, N=500, K=256, G=64, act=0, h=FAKE,
           ws=FAKE, wn=BIG, st=None, stream=None)
LORA = dict(x=FAKE, p=FAKE, s=FAKE, ids=FAKE, A=FAKE, B=FAKE, scaling=FAKE, M=300, N=500, K=256, G=64,
            n=4, R=16, y=FAKE, ws=FAKE, wn=BIG, st=None, stream=None)
FWD = dict(x=FAKE, wg=FAKE, wu=FAKE, M=300, N=500, K=256, act=0, h=FAKE, g=FAKE, u=FAKE, stream=None)
BWD = dict(dh=FAKE, x=FAKE, wg=FAKE, wu=FAKE, g=FAKE, u=FAKE, M=300, N=500, K=256, act=0, dx=FAKE,
           dwg=FAKE, dwu=FAKE, ws=FAKE, wn=BIG, stream=None)


@pytest.mark.parametrize("fn,spec,pointers", [
    ("tq_glu", GLU, ["x", "gp", "gs", "up", "us", "h"]),
    ("tq_lora_matmul", LORA, ["x", "p", "s", "ids", "A", "B", "scaling", "y"]),
    ("tq_glu_forward", FWD, ["x", "wg", "wu", "h", "g", "u"]),
    ("tq_glu_backward", BWD, ["dh", "x", "wg", "wu", "g", "u", "dx", "dwg", "dwu"])])
def test_null_pointers_and_shapes(fn, spec, pointers):
    for p in pointers:
        assert _call(fn, spec, **{p: None}) == NULL, p
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(N=-5), dict(K=100), dict(K=(1 << 22) + 256),
                dict(M=1 << 31), dict(N=1 << 31), dict(N=1 << 30, K=4096)):
        assert _call(fn, spec, **bad) == SHAPE, bad


@pytest.mark.parametrize("fn,spec", [("tq_glu", GLU), ("tq_lora_matmul", LORA)])
def test_groups(fn, spec):
    for G in (0, 32, 96, 256, -64):
        assert _call(fn, spec, G=G) == GROUP
    assert _call(fn, spec, K=192, G=128) == SHAPE


def test_activations():
    for fn, spec in (("tq_glu", GLU), ("tq_glu_forward", FWD), ("tq_glu_backward", BWD)):
        for act in (-1, 2, 99):
            assert _call(fn, spec, act=act) == ACT


def test_alignment():
    for fn, spec, by2, by4, by16 in (
            ("tq_glu", GLU, ["gs", "us", "h"], ["st"], ["x"]),
            ("tq_lora_matmul", LORA, ["s"], ["ids", "scaling", "y", "st"], ["x", "A", "B"]),
            ("tq_glu_forward", FWD, [], [], ["x", "wg", "wu", "h", "g", "u"]),
            ("tq_glu_backward", BWD, [], [], ["dh", "x", "wg", "wu", "g", "u", "dx", "dwg", "dwu"])):
        for names, off in ((by2, 1), (by4, 2), (by16, 8)):
            for n in names:
                assert _call(fn, spec, **{n: FAKE + off}) == ALIGN, (fn, n)


def test_adapters():
    for bad in (dict(R=0), dict(R=4), dict(R=12), dict(R=264), dict(R=-8), dict(n=-1), dict(n=1 << 31)):
        assert _call("tq_lora_matmul", LORA, **bad) == SHAPE, bad


def test_workspaces():
    lib = _lib()
    for fn, spec, need in (
            ("tq_glu", dict(GLU, M=4096, N=4096, K=4096), lib.tq_glu_workspace(4096, 4096, 4096, 64)),
            ("tq_lora_matmul", LORA, lib.tq_lora_workspace(300, 500, 256, 64, 16)),
            ("tq_glu_backward", BWD, lib.tq_glu_backward_workspace(300, 500, 256))):
        assert need >= 0
        if need == 0:
            continue
        assert _call(fn, spec, wn=need - 1) == WORKSPACE
        assert _call(fn, spec, wn=-1) == WORKSPACE
        assert _call(fn, spec, ws=None) == NULL
        assert _call(fn, spec, ws=FAKE + 8) == ALIGN


def test_workspace_helpers_refuse_bad_arguments():
    lib = _lib()
    assert lib.tq_glu_workspace(0, 8, 64, 64) == 0
    assert lib.tq_glu_workspace(5, 8, 100, 64) == 0
    assert lib.tq_glu_workspace(5, 8, 64, 32) == 0
    assert lib.tq_lora_workspace(5, 8, 64, 64, 7) == 0
    assert lib.tq_lora_workspace(-1, 8, 64, 64, 8) == 0
    assert lib.tq_glu_backward_workspace(4, 0, 64) == 0
    assert lib.tq_glu_backward_workspace(4, 8, 96) == 0


def test_no_rows_enqueue_nothing():
    """M = 0 is accepted with NULL activations (the backward call, which sets
    the weight gradients to 0, is checked on the GPU)."""
    assert _call("tq_glu", GLU, M=0, x=None, h=None, ws=None, wn=0) == 0
    assert _call("tq_lora_matmul", LORA, M=0, x=None, ids=None, y=None, ws=None, wn=0) == 0
    assert _call("tq_glu_forward", FWD, M=0, x=None, h=None, g=None, u=None) == 0


def test_status_strings():
    lib = _lib()
    assert b"WORKSPACE" in lib.tq_status_string(-6) and b"ACT" in lib.tq_status_string(-7)


def test_binding_refuses_host_tensors_and_unknown_activations():
    import ternary_weight_only_amd as tq
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.zeros(4, 64, dtype=torch.bfloat16)
    pair = (torch.zeros(4, 13, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.float16))
    mn = torch.zeros(2, 4, dtype=torch.bfloat16)
    for call in (lambda: tq.glu(x, pair, pair, 4, 64, 64),
                 lambda: tq.lora_matmul(x, *pair, torch.zeros(2, dtype=torch.int32), w[None], w[None],
                                        torch.ones(1), 4, 64, 64),
                 lambda: tq.glu_forward(x, w, w), lambda: tq.glu_backward(mn, x, w, w, mn, mn),
                 lambda: tq.GLU.apply(x, w, w)):
        with pytest.raises(tq.TQError):
            call()

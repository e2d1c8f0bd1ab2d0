"""Which kernels the sizes of the GPU tests run, by the library's own rules
(host only): a rule that changes must not leave a kernel untested."""
import ctypes

import pytest

from tests.test_ffn_args import _lib

FEW, MID, WIDE = 0, 1, 2
ONE, TWO = 1, 2                     # matrices: tq_lora_matmul, tq_glu


def projection(M, N, K, G, matrices, R=8):
    """(kernel, splits of K, splits of K for t, whether each block makes t, few_kernel's waves of a tile and tiles)."""
    plan = (ctypes.c_int64 * 6)()
    assert _lib().tq_probe_projection_plan(M, N, K, G, matrices, R, plan) == 0
    return tuple(plan)


def train(M, N, K):
    """(forward tile, backward tile, side by side, splits of dW, splits of dx)."""
    plan = (ctypes.c_int64 * 5)()
    assert _lib().tq_probe_train_plan(M, N, K, plan) == 0
    return tuple(plan)


def test_refusals():
    lib, plan = _lib(), (ctypes.c_int64 * 6)()
    for bad, rc in (((4, 8, 64, 32, 2, 8), -3), ((4, 8, 100, 64, 2, 8), -2), ((0, 8, 64, 64, 2, 8), -2),
                    ((4, 8, 64, 64, 3, 8), -2), ((4, 8, 64, 64, 1, 12), -2)):
        assert lib.tq_probe_projection_plan(*bad, plan) == rc, bad
    assert lib.tq_probe_projection_plan(4, 8, 64, 64, 2, 8, None) == -1
    assert lib.tq_probe_train_plan(4, 8, 96, plan) == -2 and lib.tq_probe_train_plan(0, 8, 64, plan) == -2
    assert lib.tq_probe_train_plan(4, 8, 64, None) == -1


@pytest.mark.parametrize("N,K,M", [(14336, 8192, 1), (14336, 14336, 1), (14336, 4096, 7), (3584, 1024, 1), (7168, 4096, 1), (3584, 4096, 16)])
def test_neighbouring_widths_of_few_rows_are_treated_alike(N, K, M):
    """No width is special: a tile more or less changes no waves but where it
    makes another set necessary."""
    plans = {projection(M, n, K, 128, TWO) for n in (N - 32, N - 16, N, N + 16)}
    assert len(plans) == 1, plans


def test_few_rows_use_the_block_and_few_sets():
    for M in (1, 7, 16, 24, 32):
        for K in (128, 640, 4096, 8192, 14336):
            for N in (16, 3584, 7168, 11008, 14336, 28672):
                kernel, splits, _, _, wk, wt = projection(M, N, K, 128, TWO)
                assert kernel == FEW and 1 <= wk * wt <= 16
                blocks, tiles = max(1, 256 // splits), -(-N // 16)
                assert -(-tiles // (blocks * wt)) == -(-tiles // (blocks * (16 // wk))), "a set more than the waves need"


def test_sizes_of_the_spread_tests():
    from tests import test_gpu_ffn_spread as t
    for matrices, wide in ((ONE, t.WIDE_ONE), (TWO, t.WIDE_TWO)):
        plans = {s: projection(*s, matrices) for s in t.SHAPES + wide}
        kinds = {(p[0], p[1] > 1) for p in plans.values()}
        assert kinds == {(k, split) for k in (FEW, MID, WIDE) for split in (False, True)}, plans
        assert all(plans[s][0] == WIDE for s in wide)


def test_sizes_of_the_training_tile_tests():
    from tests import test_gpu_glu_train_tiles as t
    assert all(train(*s[:3])[0] == 256 for s in t.FORWARD)
    assert [train(*s[:3])[1:] for s in t.BACKWARD] == [
        (256, 1, 1, 2), (256, 1, 1, 4), (256, 0, 1, 4), (256, 1, 4, 2), (256, 0, 8, 1), (256, 1, 1, 1)]


def test_sizes_of_the_split_and_scale_tests():
    from tests import test_gpu_lora_splits as s
    from tests import test_gpu_wide_scales as w

    def of(cases):
        return [projection(*c[:4], ONE, c[5])[:3] for c in cases]

    for cases, kernel in ((s.MANY, MID), (s.FEW, MID), (s.WIDE, WIDE), (s.LITTLE, FEW)):
        assert all(p[0] == kernel and (p[1] > 1 or kernel == FEW) for p in of(cases)), of(cases)
    assert {p[2] for p in of(s.MANY)} == {2, 4} and {p[2] for p in of(s.LITTLE)} == {1, 2}
    assert all(projection(*c, TWO)[0] == WIDE for c in w.GLU) and all(projection(*c, ONE)[0] == WIDE for c in w.LORA)
    assert {projection(*c, TWO)[0] for c in w.LONG} == {FEW, MID, WIDE}

"""Which kernels the products of 8-bit rows run (a host-only query), and that the
GPU tests' sizes reach every one of them, with and without splits of K."""
import ctypes
import os

import pytest

import ternary_weight_only_amd as tq
from tests.i8_reference import LARGE, MIDDLE


def plan(M, N, K, G, E=0):
    if not os.path.exists(tq.binding.LIB_PATH):
        from ternary_weight_only_amd import build
        build.build_library()
    got = (ctypes.c_int64 * 7)()
    assert tq.lib().tq_probe_i8_plan(M, N, K, G, E, ctypes.cast(got, ctypes.c_void_p)) == 0
    return list(got)


def test_the_gpu_tests_sizes_reach_every_kernel():
    few, tiles = set(), set()
    for M, N, K, G, E in MIDDLE + LARGE:
        p = plan(M, N, K, G, E)
        if p[0] == 0:
            few.add((G, p[2], p[3]))
        else:
            tiles.add((G, p[0], p[2], p[3], p[1] > 1))
    assert few == {(G, rows, copies) for G in (64, 128) for rows in (4, 8, 16) for copies in (8, 32)}
    both = {(64, 1, 128, 64), (64, 1, 128, 128), (64, 1, 256, 256), (128, 1, 128, 64), (128, 1, 128, 128),
            (128, 2, 256, 256)}
    assert tiles == {t + (split,) for t in both for split in (False, True)}


def test_the_gpu_tests_sizes_take_more_than_one_round():
    """Blocks that go on to a second tile, of every shape, and with splits."""
    again = set()
    for M, N, K, G, E in LARGE:
        p = plan(M, N, K, G, E)
        units = M // p[3] + E // 2 if E else -(-M // p[3])
        if units * -(-N // p[2]) * p[1] > (256 if p[2] == 256 else 512):
            again.add((G, p[2], p[3], p[1] > 1))
    assert {(G, *shape, False) for G in (64, 128) for shape in ((128, 64), (128, 128), (256, 256))} <= again
    assert (128, 256, 256, True) in again


def test_the_gpu_tests_sizes_take_many_sets_of_a_block():
    """Blocks that go on to a second set of tiles, at every number of rows of a unit."""
    again = set()
    for M, N, K, G, E in MIDDLE:
        p = plan(M, N, K, G, E)
        if p[0] == 0 and -(-N // (16 * p[5])) * p[1] > p[6]:
            again.add((G, p[2], p[3]))
    assert {(G, rows, 32) for G in (64, 128) for rows in (4, 8, 16)} <= again
    assert (64, 16, 8) in again and (128, 16, 8) in again


def test_few_rows_in_many_shapes_of_blocks():
    """Waves of a tile and tiles of a set both vary; q's rows fit at any K."""
    shapes = {tuple(plan(M, N, K, 128, E)[4:6]) for M in (1, 7, 16) for N in (16, 700, 14336)
              for K in (128, 3584, 14336) for E in (0, 8)}
    assert len(shapes) > 6
    for E in (0, 3, 32768):
        for K in (1 << 21, 1 << 20, 14336):
            p = plan(16, 16, K, 128, E)
            assert p[0] == 0 and p[1] >= 1 and p[4] * p[5] <= 16


def test_launches_stay_within_a_launch():
    """Blocks times threads stay below 2^32 at the largest sizes."""
    for M, N, K, E in ((1 << 19, 8, 1 << 21, 65535), (1 << 30, 1024, 64, 65536), (1 << 19, 8, 1 << 21, 65536),
                       (8, 8, 1 << 21, 65536), (1 << 30, 1024, 64, 0), (1, 1 << 30, 64, 0), (16, 1 << 19, 1 << 21, 0)):
        p = plan(M, N, K, 64, E)
        if p[0] == 0:
            units = M // p[2] + min(E, M) if E else 1
            assert units * p[1] <= p[6] and p[6] * 64 * p[4] * p[5] < 1 << 32, (M, N, K, E)


def test_refusals():
    lib = tq.lib()
    got = ctypes.cast((ctypes.c_int64 * 7)(), ctypes.c_void_p)
    for bad, rc in (((4, 8, 64, 32, 0), -3), ((4, 8, 100, 64, 0), -2), ((0, 8, 64, 64, 0), -2), ((4, 0, 64, 64, 0), -2),
                    ((4, 8, 64, 64, -1), -2), ((4, 8, 64, 64, 65537), -2)):
        assert lib.tq_probe_i8_plan(*bad, got) == rc, bad
    assert lib.tq_probe_i8_plan(4, 8, 64, 64, 0, None) == -1


@pytest.mark.parametrize("M,N,K,G,E", LARGE)
def test_workspaces_hold_the_parts_and_the_sums(M, N, K, G, E):
    p = plan(M, N, K, G, E)
    lib = tq.lib()
    have = lib.tq_expert_gemm_i8_workspace(M, N, K, G, E) if E else lib.tq_gemm_i8_workspace(M, N, K, G)
    assert have >= (M * K * 3 // 2 if p[0] == 2 else 0) + (p[1] * M * N * 4 if p[1] > 1 else 0)

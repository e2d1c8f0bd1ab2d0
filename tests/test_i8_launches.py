"""The launches of the 8-bit products at the largest sizes, for every kernel (a
host-only query)."""
import pytest

from tests.i8_reference import LARGE, MIDDLE
from tests.test_i8_plans import plan

# (rows, N, K, G, experts or 0): as many rows, columns, experts and splits of K as the calls take
LARGEST = [(1 << 19, 8, 1 << 21, 64, 65535), (1 << 30, 1024, 64, 64, 65536), (1 << 19, 8, 1 << 21, 64, 65536),
           (8, 8, 1 << 21, 64, 65536), (1 << 30, 1024, 64, 64, 0), (1, 1 << 30, 64, 64, 0), (16, 1 << 19, 1 << 21, 64, 0),
           (1 << 30, 1024, 128, 128, 65536), (1 << 30, 1024, 128, 128, 0), (17, 1 << 30, 128, 128, 0),
           (1 << 30, 1, 64, 64, 0), (17, 1 << 19, 1 << 21, 128, 0), (1 << 19, 8, 1 << 21, 128, 65536)]


@pytest.mark.parametrize("M,N,K,G,E", LARGEST + MIDDLE + LARGE)
def test_blocks_times_threads_stay_below_a_launch(M, N, K, G, E):
    p = plan(M, N, K, G, E)
    threads = 64 * p[4] * p[5] if p[0] == 0 else 2 * p[2]
    assert p[6] >= 1 and p[6] * threads < 1 << 32
    units = -(-M // p[2 if p[0] == 0 else 3])
    if p[0] == 0:  # a block at least for every unit and split
        assert (M // p[2] + min(E, M) if E else units) * p[1] <= p[6]
    elif not E:  # blocks go on to other tiles: none without one
        assert p[6] <= units * -(-N // p[2]) * p[1]


def test_the_largest_sizes_reach_every_kind():
    assert {plan(*c)[0] for c in LARGEST} == {0, 1, 2}

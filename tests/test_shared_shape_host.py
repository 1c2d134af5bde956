"""The length of the shared decode's prefix splits, as the workspace's size
shows it: against the rule tried at every length.  CPU only."""
import random
import time

import pytest

from tests.test_cache_ops_host import L  # noqa: F401

SMS, KEYS, SPLIT_COST = 152, 128, 4


def _splits(units, max_prefix):
    """Splits of the longest prefix: the length (in key tiles) with the smallest
    sum over the busiest SM's items, the longest of equals."""
    tiles = -(-max_prefix // KEYS)
    cost = lambda n: -(-units * -(-tiles // n) // SMS) * (n + SPLIT_COST)  # noqa: E731
    best = min(range(tiles, 0, -1), key=cost)
    return -(-max_prefix // (best * KEYS))


def _align(n):
    return (n + 255) // 256 * 256


@pytest.fixture
def once(L):  # noqa: F811
    import paged_kv_decode_26_gb300 as pkv
    pkv.set_tuning(shared_prefix=1)
    yield pkv.decode_shared_workspace_bytes
    pkv.reset_tuning()


def test_split_lengths(once):
    r = random.Random(3)
    for _ in range(400):
        Hk, G, D = r.choice([1, 2, 8, 32]), r.choice([1, 2, 4, 8]), r.choice([64, 128])
        S = r.randint(1, 400)
        max_group, groups = r.randint(1, S), r.choice([1, 2, 7, 16, 100, 5000])
        max_prefix = 16 * r.randint(1, r.choice([10, 1000, 9000]))
        L_max = max_prefix + r.randint(0, 500)
        units = groups * Hk * -(-max_group // (256 // G))
        rows = S * G * Hk * _splits(units, max_prefix)
        got = once(S, groups, max_group, max_prefix, G * Hk, Hk, D, 16, L_max)
        without = once(S, groups, max_group, 0, G * Hk, Hk, D, 16, L_max)
        assert got - without == _align(rows * D * 4) + _align(rows * 8), (S, groups, max_group,
                                                                          max_prefix, G, Hk, D)


def test_bounds_cost_no_time(once):
    """A bound of 2^30 tokens takes the time of a short one (it took 0.1 s)."""
    def best():
        times = []
        for _ in range(5):
            t = time.perf_counter()
            assert once(8, 1, 8, 2 ** 30, 8, 8, 64, 16, 2 ** 30) > 0
            times.append(time.perf_counter() - t)
        return min(times)
    assert best() < 0.01

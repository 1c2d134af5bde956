"""The eviction's selection by clusters of 2, 4 and 8 CTAs, with weights that
repeat so that the last one kept is a tie within a later CTA, and by single CTAs
that own more tokens than their shared memory holds: exact."""
import pytest
import torch

from tests.test_cache_ops_gpu import BF, F32, FP, _evict_case, _lognormal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [8200, 9001, 16385, 17003, 32800, 33333])
@pytest.mark.parametrize("values", [1, 3])
def test_ties_across_a_cluster(n, values):
    """values = 1: all weights equal; 3: few values, the middle one cut."""
    g = torch.Generator().manual_seed(n)
    w = torch.randint(values, (2, n + 2), generator=g).float() if values > 1 else torch.ones(2, n + 2)
    for keep, recent in ((n // 2, 0), (n // 2 + 1, 700), (n - 1, 5), (17, 16), (n * 7 // 8, 1)):
        _evict_case([n, n - 300], keep, recent, 1, 64, 16, FP, w)


@pytest.mark.parametrize("n", [9001, 17003, 33333])
def test_distinct_weights_by_a_cluster(n):
    w = _lognormal(3, n)
    w[1, ::3] = float("nan")
    w[2] = -w[2]
    _evict_case([n, n - 1, n // 2], n // 3, n // 30, 2, 64, 16, BF, w)


def test_more_tokens_than_a_cta_holds():
    """80 sequences, a CTA each: the long one's keys are read from memory again."""
    lens = [5 + i % 17 for i in range(80)]
    lens[37] = 60000
    w = _lognormal(80, 60000)
    w[37, 1000::7] = 0.25
    _evict_case(lens, 9000, 100, 1, 4, 16, F32, w)
    w[37] = 2.0
    _evict_case(lens, 59999, 0, 1, 4, 16, F32, w)

"""Sizes at the end of what the cache operators' 32-bit arithmetic holds, and
arguments that lie on one another.  CPU only: refused before a device is
touched."""
import ctypes as C

import pytest
import torch

from tests.test_cache_ops_host import FAKE, L, NULL, _evict, _ints  # noqa: F401

MOST = 2 ** 31 - 2 ** 14


@pytest.mark.parametrize("kw", [
    # contexts that the tables and the weights allow
    dict(B=16, mb=2 ** 27 - 1, ws=2 ** 31 - 16, wc=2 ** 31 - 16),
    dict(B=16, mb=2 ** 27 - 1, ws=MOST + 1, wc=MOST + 1),
    # columns behind the staying tokens
    dict(nwc=MOST + 1, nws=MOST + 1),
    # tokens that stay
    dict(keep=MOST + 1, recent=0, nwc=MOST + 1, nws=MOST + 1, nbs=2 ** 27 - 1),
])
def test_evict_refuses_sizes_near_2_to_31(L, kw):  # noqa: F811
    assert _evict(L, **kw) == 2
    assert b"2^31 - 2^14" in L.pkv_last_error_detail()

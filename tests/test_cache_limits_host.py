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


def _manager(L):  # noqa: F811
    import paged_kv_decode_26_gb300 as pkv
    return pkv.BlockManager(12, 4, free_ids=[6, 7, 8, 9])


@pytest.mark.parametrize("new,width,old", [
    ("tables", 3, "old"),               # the tables in place
    (("tables", 4), 2, "old"),
    ("lens", 1, "old"),
    ("new", 3, "tables"),
    ("new", 3, "new"),
])
def test_evict_tables_refuses_outputs_on_inputs(L, new, width, old):  # noqa: F811
    """In place, the old ids would be read after the new ones are written: the
    caller would free the pages that it has just got."""
    bm = _manager(L)
    buf = {"tables": _ints([[0, 1, 2], [3, 4, 5]]), "lens": _ints([9, 12]),
           "new": torch.full((2, 3), -7, dtype=torch.int32),
           "old": torch.full((6,), -7, dtype=torch.int32)}
    before = {k: v.clone() for k, v in buf.items()}
    def at(x):
        name, offset = x if isinstance(x, tuple) else (x, 0)
        return C.c_void_p(buf[name].data_ptr() + offset)
    n = C.c_int(-1)
    st = L.pkv_evict_tables(bm._h, at("tables"), 3, at("lens"), 2, 4, at(new), width, at(old), 6,
                            C.byref(n))
    assert st == 1 and n.value == 0
    assert all(torch.equal(buf[k], before[k]) for k in buf)
    assert bm.free_ids() == [6, 7, 8, 9]

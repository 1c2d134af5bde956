"""Refusals of the copy of an 8-bit cache's scales.  CPU only: every refused call fails
validation before a device is touched."""
import ctypes as C

import pytest

from paged_kv_decode_26_gb300 import build

NULL, FAKE = C.c_void_p(0), C.c_void_p(4096)      # never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    from paged_kv_decode_26_gb300._lib import lib
    return lib()


@pytest.mark.parametrize("kw,code", [
    (dict(hk=0), 1), (dict(hk=-1), 1), (dict(n=-1), 1), (dict(ns=-1), 1), (dict(nd=-1), 1),
    (dict(dk=NULL), 1), (dict(sk=NULL), 1), (dict(dv=NULL), 1), (dict(sv=NULL), 1),
    (dict(pairs=NULL), 1), (dict(pairs=C.c_void_p(4100)), 1), (dict(dk=C.c_void_p(4098)), 1),
    (dict(sv=C.c_void_p(4097)), 1), (dict(n=0), 0), (dict(n=0, dv=NULL, sv=NULL), 0),
])
def test_refusals(L, kw, code):
    a = dict(dk=FAKE, dv=FAKE, sk=FAKE, sv=FAKE, hk=3, pairs=FAKE, n=1, ns=4, nd=4)
    a.update(kw)
    assert L.swap_block_scales(a["dk"], a["dv"], a["sk"], a["sv"], a["hk"], a["pairs"], a["n"], a["ns"],
                               a["nd"], NULL) == code
    assert code == 0 or L.pkv_last_error_detail()

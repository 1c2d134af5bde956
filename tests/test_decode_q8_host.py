"""Refusals and workspace sizes of the attention over 8-bit pages.  CPU only:
every refused call fails validation before a device is touched."""
import ctypes as C

import pytest

from paged_kv_decode_26_gb300 import build

NULL = C.c_void_p(0)
MB = 1 << 20


def FAKE(i=1):
    return C.c_void_p(i * 64 * MB)      # never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    from paged_kv_decode_26_gb300._lib import lib
    return lib()


def _decode(L, **kw):
    a = dict(out=FAKE(1), od=1, q=FAKE(2), qd=1, k=FAKE(3), v=FAKE(4), ks=FAKE(5), vs=FAKE(6),
             bt=FAKE(7), mb=4, cl=FAKE(8), S=2, H=8, Hk=8, D=128, B=16, nb=10, scale=0.1, maxc=64,
             ws=FAKE(9), wsb=0)
    a.update(kw)
    return L.paged_attn_decode_q8(a["out"], a["od"], a["q"], a["qd"], a["k"], a["v"], a["ks"],
                                  a["vs"], a["bt"], a["mb"], a["cl"], a["S"], a["H"], a["Hk"],
                                  a["D"], a["B"], a["nb"], a["scale"], a["maxc"], a["ws"],
                                  a["wsb"], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(S=65536), 2), (dict(maxc=-1), 1), (dict(H=6, Hk=4), 1),
    (dict(D=96), 2), (dict(B=8), 2), (dict(H=48, Hk=4), 2), (dict(H=8192, Hk=8192), 2),
    (dict(qd=2), 2), (dict(od=7), 1), (dict(nb=-1), 1), (dict(k=NULL), 1), (dict(mb=0), 1),
    (dict(scale=float("nan")), 1), (dict(q=NULL), 1), (dict(cl=NULL), 1), (dict(ks=NULL), 1),
    (dict(vs=NULL), 1), (dict(ks=C.c_void_p(4098)), 1), (dict(out=C.c_void_p(4104)), 1),
    (dict(v=C.c_void_p(4104)), 1), (dict(mb=1 << 27, B=32), 2),
    (dict(S=65535, maxc=1 << 30, mb=1 << 26), 2),
])
def test_decode_refusals(L, kw, code):
    assert _decode(L, **kw) == code
    assert L.pkv_last_error_detail()


def test_decode_of_no_sequences_is_a_no_op(L):
    assert _decode(L, S=0, q=NULL, ks=NULL) == 0


def test_decode_workspace_bytes(L):
    f = L.pkv_decode_q8_workspace_bytes
    assert f(2, 8, 3, 128, 16, 100) == 0 and f(0, 8, 8, 128, 16, 100) == 0
    # few short contexts are decoded whole
    assert f(2, 8, 8, 128, 16, 100) == 0
    # else at least a partial row per (sequence, head)
    assert f(2, 8, 8, 128, 16, 5000) >= 2 * 8 * (128 + 2) * 4
    assert f(3, 8, 8, 128, 16, 5000) > f(2, 8, 8, 128, 16, 5000)


def _chunk(L, **kw):
    a = dict(out=FAKE(1), od=1, q=FAKE(2), qd=1, qs=FAKE(10), T=8, maxq=4, k=FAKE(3), v=FAKE(4),
             ks=FAKE(5), vs=FAKE(6), bt=FAKE(7), mb=4, cl=FAKE(8), S=2, H=8, Hk=8, D=128, B=16,
             nb=10, scale=0.1, maxc=64, ws=NULL, wsb=0)
    a.update(kw)
    return L.paged_attn_multi_query_q8(a["out"], a["od"], a["q"], a["qd"], a["qs"], a["T"],
                                       a["maxq"], a["k"], a["v"], a["ks"], a["vs"], a["bt"],
                                       a["mb"], a["cl"], a["S"], a["H"], a["Hk"], a["D"], a["B"],
                                       a["nb"], a["scale"], a["maxc"], a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(S=65536), 2), (dict(T=-1), 1), (dict(maxq=-1), 1), (dict(maxc=-1), 1),
    (dict(H=6, Hk=4), 1), (dict(D=96), 2), (dict(B=8), 2), (dict(H=48, Hk=4), 2), (dict(qd=2), 2),
    (dict(od=7), 1), (dict(nb=-1), 1), (dict(k=NULL), 1), (dict(mb=0), 1),
    (dict(scale=float("inf")), 1), (dict(q=NULL), 1), (dict(qs=NULL), 1),
    (dict(qs=C.c_void_p(4098)), 1), (dict(cl=NULL), 1), (dict(ks=NULL), 1), (dict(vs=NULL), 1),
    (dict(vs=C.c_void_p(4098)), 1), (dict(out=C.c_void_p(4104)), 1), (dict(v=C.c_void_p(4104)), 1),
    (dict(mb=1 << 27, B=32), 2),
])
def test_chunk_refusals(L, kw, code):
    assert _chunk(L, **kw) == code
    assert L.pkv_last_error_detail()


@pytest.mark.parametrize("kw", [dict(S=0), dict(T=0), dict(maxq=0)])
def test_chunk_of_nothing_is_a_no_op(L, kw):
    assert _chunk(L, q=NULL, ks=NULL, **kw) == 0


def test_chunk_workspace_bytes(L):
    f = L.pkv_multi_query_q8_workspace_bytes
    assert f(2, 64, 8, 3, 128, 16, 5000) == 0 and f(0, 64, 8, 8, 128, 16, 5000) == 0
    # too few keys to cut
    assert f(64, 256, 32, 32, 128, 16, 500) == 0 and f(1, 16, 8, 8, 128, 16, 200) == 0
    # one pair of row tiles: parts of every row; many: only of what fills no round of its own
    assert f(1, 16, 1, 1, 128, 16, 5000) >= 2 * 256 * (128 + 2) * 4
    assert f(64, 2560, 32, 32, 128, 16, 50000) < 1 << 28

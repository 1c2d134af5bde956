"""Refusals and host bookkeeping of the cache-budget calls.  CPU only: every
refused call fails validation before a device is touched."""
import ctypes as C

import pytest
import torch

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


def _weights(L, **kw):
    a = dict(out=FAKE(1), od=1, q=FAKE(2), k=FAKE(3), v=FAKE(4), kd=1, bt=FAKE(5), mb=4,
             cl=FAKE(6), w=FAKE(7), ws_=64, S=2, H=8, Hk=8, D=128, B=16, nb=10, scale=0.1, maxc=64,
             ws=FAKE(8), wsb=0)
    a.update(kw)
    return L.paged_attn_decode_weights(
        a["out"], a["od"], a["q"], a["k"], a["v"], a["kd"], a["bt"], a["mb"], a["cl"], a["w"],
        a["ws_"], a["S"], a["H"], a["Hk"], a["D"], a["B"], a["nb"], a["scale"], a["maxc"],
        a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(S=65536), 2), (dict(maxc=-1), 1), (dict(H=6, Hk=4), 1),
    (dict(D=96), 2), (dict(B=8), 2), (dict(H=48, Hk=4), 2), (dict(H=8192, Hk=8192), 2),
    (dict(kd=2), 2), (dict(od=7), 1), (dict(nb=-1), 1), (dict(k=NULL), 1), (dict(mb=0), 1),
    (dict(scale=float("inf")), 1), (dict(q=NULL), 1), (dict(cl=NULL), 1), (dict(w=NULL), 1),
    (dict(ws_=63), 1), (dict(w=C.c_void_p(4098)), 1), (dict(out=C.c_void_p(4104)), 1),
    (dict(mb=1 << 27, B=32), 2), (dict(S=65535, maxc=1 << 30, mb=1 << 26, ws_=1 << 30), 2),
])
def test_weights_refusals(L, kw, code):
    assert _weights(L, **kw) == code
    assert L.pkv_last_error_detail()


def test_weights_of_no_sequences_is_a_no_op(L):
    assert _weights(L, S=0, q=NULL, w=NULL) == 0


def test_weights_workspace_bytes(L):
    f = L.pkv_decode_weights_workspace_bytes
    assert f(2, 8, 3, 128, 16, 100) == 0 and f(0, 8, 8, 128, 16, 100) == 0
    # at least the scores of every head and token, and it grows with each
    assert f(2, 8, 8, 128, 16, 100) >= 2 * 8 * 112 * 4
    assert f(3, 8, 8, 128, 16, 100) > f(2, 8, 8, 128, 16, 100)
    assert f(2, 8, 8, 128, 16, 5000) > f(2, 8, 8, 128, 16, 100)


def _evict(L, **kw):
    a = dict(k=FAKE(1), v=FAKE(2), dt=1, bt=FAKE(3), mb=4, cl=FAKE(4), w=FAKE(5), ws=64, wc=64,
             nt=FAKE(6), nbs=2, nl=FAKE(7), nw=FAKE(8), nws=32, nwc=32, kept=FAKE(9), S=2,
             keep=32, recent=8, Hk=8, D=128, B=16, nb=10)
    a.update(kw)
    return L.kv_evict(a["k"], a["v"], a["dt"], a["bt"], a["mb"], a["cl"], a["w"], a["ws"], a["wc"],
                      a["nt"], a["nbs"], a["nl"], a["nw"], a["nws"], a["nwc"], a["kept"], a["S"],
                      a["keep"], a["recent"], a["Hk"], a["D"], a["B"], a["nb"], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(S=65536), 2), (dict(keep=0), 1), (dict(recent=-1), 1),
    (dict(recent=33), 1), (dict(keep=33, nwc=40, nws=40), 1), (dict(ws=63), 1), (dict(nws=31), 1),
    (dict(nwc=31), 1), (dict(dt=5), 1), (dict(Hk=1, D=4), 2), (dict(Hk=0), 1), (dict(B=0), 1),
    (dict(mb=0), 1), (dict(nb=-1), 1), (dict(k=NULL), 1), (dict(kept=NULL), 1),
    (dict(k=C.c_void_p(4104)), 1), (dict(mb=1 << 28), 2),
    (dict(nl=FAKE(4)), 1),                                  # the lengths in place
    (dict(nw=C.c_void_p(5 * 64 * MB + 256)), 1),            # the weights in place
    (dict(kept=FAKE(6)), 1),
])
def test_evict_refusals(L, kw, code):
    assert _evict(L, **kw) == code
    assert L.pkv_last_error_detail()


def test_evict_of_no_sequences_is_a_no_op(L):
    assert _evict(L, S=0, w=NULL) == 0


def _ints(x):
    return torch.tensor(x, dtype=torch.int32)


def test_evict_tables(L):
    import paged_kv_decode_26_gb300 as pkv
    bm = pkv.BlockManager(12, 4, free_ids=[1, 4, 6, 7, 9])
    bm.add_reference(0)                          # a page two sequences share
    tables = _ints([[0, 2, 3, 5], [0, 8, -1, -1], [10, 11, -1, -1], [-1, -1, -1, -1]])
    lens = _ints([14, 8, 5, 0])
    new, old = bm.evict_tables(tables, lens, 6, new_blocks_per_seq=3)
    assert new.tolist() == [[1, 4, -1], [6, 7, -1], [10, 11, -1], [-1, -1, -1]]
    assert lens.tolist() == [6, 6, 5, 0] and old.tolist() == [0, 2, 3, 5, 0, 8]
    assert bm.free_ids() == [9] and bm.ref_count(0) == 2
    for b in old.tolist():
        bm.free(b)
    assert bm.free_ids() == [0, 2, 3, 5, 8, 9] and bm.ref_count(0) == 0


@pytest.mark.parametrize("lens,keep,width,free,status", [
    ([9, 9], 5, 3, [7], 5),           # too few free blocks: nothing changes
    ([9, 9], 5, 1, [6, 7], 1),        # a row that does not fit
    ([3, 13], 5, 3, [6, 7], 1),       # a length beyond the table
    ([3, -1], 5, 3, [6, 7], 1),
])
def test_evict_tables_refuses_and_changes_nothing(L, lens, keep, width, free, status):
    import paged_kv_decode_26_gb300 as pkv
    bm = pkv.BlockManager(8, 4, free_ids=free)
    tables, n = _ints([[0, 1, 2], [3, 4, 5]]), _ints(lens)
    with pytest.raises(pkv.PagedKVError) as e:
        bm.evict_tables(tables, n, keep, new_blocks_per_seq=width)
    assert e.value.status == status
    assert n.tolist() == lens and bm.free_ids() == free


def test_evict_tables_refuses_unheld_pages(L):
    import paged_kv_decode_26_gb300 as pkv
    bm = pkv.BlockManager(8, 4, free_ids=[1, 6, 7])
    with pytest.raises(pkv.PagedKVError):
        bm.evict_tables(_ints([[0, 1, 2]]), _ints([9]), 5)
    with pytest.raises(pkv.PagedKVError):
        bm.evict_tables(_ints([[0, -1, 2]]), _ints([9]), 5)
    with pytest.raises(ValueError):
        bm.evict_tables(_ints([[0, 2]]).long(), _ints([9]), 5)


def _prompt(L, **kw):
    a = dict(out=FAKE(1), od=1, q=FAKE(2), qs=1024, k=FAKE(3), ks=256, v=FAKE(4), vs=256, dt=1,
             st=FAKE(5), S=2, T=100, ml=60, H=8, Hk=2, D=128, scale=0.1)
    a.update(kw)
    return L.pkv_attn_prompt(a["out"], a["od"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                         a["dt"], a["st"], a["S"], a["T"], a["ml"], a["H"], a["Hk"], a["D"],
                         a["scale"], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(T=-1), 1), (dict(ml=-1), 1), (dict(H=6, Hk=4), 1), (dict(D=96), 2),
    (dict(H=6), 2), (dict(dt=2), 2), (dict(od=9), 1), (dict(scale=float("nan")), 1),
    (dict(qs=1016), 1), (dict(ks=255), 1), (dict(vs=260), 1), (dict(vs=1 << 40), 2),
    (dict(q=NULL), 1), (dict(out=NULL), 1), (dict(st=NULL), 1), (dict(k=C.c_void_p(4104)), 1),
    (dict(st=C.c_void_p(4097)), 1), (dict(S=1 << 30, H=8, Hk=8, ks=1024, vs=1024), 2),
])
def test_prompt_refusals(L, kw, code):
    assert _prompt(L, **kw) == code
    assert L.pkv_last_error_detail()


@pytest.mark.parametrize("kw", [dict(S=0, st=NULL), dict(T=0, q=NULL), dict(ml=0)])
def test_prompt_of_nothing_is_a_no_op(L, kw):
    assert _prompt(L, **kw) == 0


def _shared(L, **kw):
    a = dict(out=FAKE(1), od=1, q=FAKE(2), k=FAKE(3), v=FAKE(4), kd=1, bt=FAKE(5), mb=4,
             cl=FAKE(6), gs=FAKE(7), pl=FAKE(8), ng=1, mg=2, mp=32, S=2, H=8, Hk=8, D=128, B=16,
             nb=10, scale=0.1, maxc=64, ws=FAKE(9), wsb=0)
    a.update(kw)
    return L.paged_attn_decode_shared(
        a["out"], a["od"], a["q"], a["k"], a["v"], a["kd"], a["bt"], a["mb"], a["cl"], a["gs"],
        a["pl"], a["ng"], a["mg"], a["mp"], a["S"], a["H"], a["Hk"], a["D"], a["B"], a["nb"],
        a["scale"], a["maxc"], a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(S=65536), 2), (dict(ng=-1), 1), (dict(ng=65536), 2), (dict(mg=-1), 1),
    (dict(mg=3), 1), (dict(mp=-1), 1), (dict(mp=65), 1), (dict(gs=NULL), 1), (dict(pl=NULL), 1),
    (dict(gs=C.c_void_p(4098)), 1), (dict(H=6, Hk=4), 1), (dict(D=96), 2), (dict(B=8), 2),
    (dict(kd=2), 2), (dict(od=7), 1), (dict(k=NULL), 1), (dict(scale=float("nan")), 1),
    (dict(q=NULL), 1), (dict(out=C.c_void_p(4104)), 1),
])
def test_shared_refusals(L, kw, code):
    assert _shared(L, **kw) == code
    assert L.pkv_last_error_detail()


def test_shared_of_no_sequences_is_a_no_op(L):
    assert _shared(L, S=0, mg=0, q=NULL) == 0


def test_shared_workspace_bytes(L):
    f = L.pkv_decode_shared_workspace_bytes
    assert f(4, 1, 5, 64, 8, 8, 128, 16, 100) == 0          # a group beyond the batch
    assert f(4, 1, 4, 101, 8, 8, 128, 16, 100) == 0         # a prefix beyond the context
    assert f(4, 0, 0, 0, 8, 8, 128, 16, 100) > 0
    assert f(64, 1, 64, 4096, 8, 8, 128, 16, 5000) > f(64, 0, 0, 0, 8, 8, 128, 16, 5000)


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_tensors_that_are_not_on_the_gpu(L):
    """Checked before anything touches a device."""
    import paged_kv_decode_26_gb300 as pkv
    out, q = _cpu(2, 4, 64), _cpu(2, 4, 64)
    pool, tables, lens = _cpu(4, 16, 2, 64), _ints([[0, 1], [2, 3]]), _ints([20, 30])
    w = torch.zeros(2, 32)
    for call in (
            lambda: pkv.attn_prompt(out, q, q[:, :2], q[:, :2], _ints([0, 2]), 0.1, 2),
            lambda: pkv.paged_attn_decode_weights(out, q, pool, pool, tables, lens, w, 0.1, 32),
            lambda: pkv.paged_attn_decode_shared(out, q, pool, pool, tables, lens, _ints([0, 2]),
                                                 _ints([16]), 0.1, 32, 2, 16),
            lambda: pkv.kv_evict(pool, pool, tables, lens, w, tables, lens.clone(), w.clone(),
                                 _ints([[0] * 8] * 2), 8, 2)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


ODD = C.c_void_p(30 * 64 * MB + 2)


@pytest.mark.parametrize("call,name", [
    (_weights, "bt"), (_weights, "cl"), (_shared, "bt"), (_shared, "cl"), (_shared, "pl"),
    (_evict, "bt"), (_evict, "cl"), (_evict, "w"), (_evict, "nt"), (_evict, "nl"),
    (_evict, "nw"), (_evict, "kept")])
def test_refuses_misaligned_ints_and_weights(L, call, name):
    assert call(L, **{name: ODD}) == 1
    assert b"4-byte" in L.pkv_last_error_detail()


@pytest.mark.parametrize("kw", [
    dict(kept=FAKE(8)), dict(nl=FAKE(9)), dict(nl=FAKE(8)),
    dict(kept=C.c_void_p(8 * 64 * MB + 128)), dict(nl=C.c_void_p(9 * 64 * MB + 252))])
def test_evict_refuses_outputs_that_overlap(L, kw):
    assert _evict(L, **kw) == 1
    assert b"overlap" in L.pkv_last_error_detail()

"""Refusals of the rotating appends and their frequencies.  CPU only: every
refused call fails validation before a device is touched."""
import ctypes as C
import math

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


def _call(L, q8, **kw):
    a = dict(kp=FAKE(1), vp=FAKE(2), ksc=FAKE(3), vsc=FAKE(4), k=FAKE(5), k_s=1024, v=FAKE(6),
             v_s=1024, dt=1, slots=FAKE(7), pos=FAKE(8), table=FAKE(9), rows=100, rot=64, inter=0,
             q=FAKE(10), q_s=1024, qo=FAKE(11), qo_s=1024, ko=FAKE(12), ko_s=1024, T=10, H=8, Hk=8,
             D=128, B=16, nb=10)
    a.update(kw)
    scales = [a["ksc"], a["vsc"]] if q8 else []
    fn = L.kv_append_rope_q8 if q8 else L.kv_append_rope
    return fn(a["kp"], a["vp"], *scales, a["k"], a["k_s"], a["v"], a["v_s"], a["dt"], a["slots"],
              a["pos"], a["table"], a["rows"], a["rot"], a["inter"], a["q"], a["q_s"], a["qo"],
              a["qo_s"], a["ko"], a["ko_s"], a["T"], a["H"], a["Hk"], a["D"], a["B"], a["nb"],
              NULL)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(Hk=0), 1), (dict(H=-1), 1), (dict(nb=-1), 1), (dict(dt=2), 2),
    (dict(D=96), 2), (dict(Hk=5000), 2), (dict(H=5000), 2), (dict(rot=0), 1), (dict(rot=24), 1),
    (dict(rot=144), 1), (dict(rows=-1), 1), (dict(table=C.c_void_p(4100)), 1),
    (dict(table=NULL), 1), (dict(qo=NULL), 1), (dict(q=NULL), 1), (dict(H=0), 1),
    (dict(slots=NULL), 1), (dict(kp=NULL), 1), (dict(vp=NULL), 1), (dict(pos=NULL), 1),
    (dict(k=NULL), 1), (dict(v=NULL), 1), (dict(kp=C.c_void_p(4104)), 1),
    (dict(slots=C.c_void_p(4100)), 1), (dict(pos=C.c_void_p(4098)), 1),
    (dict(k=C.c_void_p(4104)), 1), (dict(k_s=1016), 1), (dict(k_s=1028), 1), (dict(v_s=512), 1),
    (dict(q_s=1000), 1), (dict(qo_s=8), 1), (dict(ko_s=1032 - 16), 1), (dict(k_s=1 << 41), 2),
    (dict(vp=FAKE(1)), 1), (dict(qo=FAKE(5)), 1), (dict(qo=FAKE(6)), 1), (dict(ko=FAKE(6)), 1),
    (dict(ko=FAKE(10)), 1), (dict(qo=FAKE(10), qo_s=2048), 1), (dict(ko=FAKE(11)), 1),
    (dict(qo=FAKE(1)), 1), (dict(k=FAKE(2)), 1), (dict(B=0), None),
])
def test_refusals(L, q8, kw, code):
    got = _call(L, q8, **kw)
    assert got == code if code else got in (1, 2)
    assert L.pkv_last_error_detail()


@pytest.mark.parametrize("kw,code", [
    (dict(B=8), 2), (dict(B=64), 2), (dict(ksc=NULL), 1), (dict(vsc=NULL), 1),
    (dict(ksc=C.c_void_p(4098)), 1), (dict(vsc=FAKE(3)), 1),
])
def test_scale_refusals(L, kw, code):
    assert _call(L, True, **kw) == code
    assert L.pkv_last_error_detail()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw", [
    dict(ko=FAKE(5), v=FAKE(5)),                           # keys in place that are the values too
    dict(qo=FAKE(10), q_s=2048, qo_s=2048, k=C.c_void_p(640 * MB + 1024), k_s=2048),
    dict(qo=FAKE(10), q_s=2048, qo_s=2048, k=C.c_void_p(640 * MB + 2048), k_s=4096),
    dict(qo=FAKE(10), ko=FAKE(10), k=FAKE(10)),            # both in place, in the same rows
])
def test_refusals_in_place(L, q8, kw):
    """What is rotated in place lies beside the other inputs, not over them."""
    assert _call(L, q8, **kw) == 1
    assert L.pkv_last_error_detail()


def test_scales_in_a_pool(L):
    for kw in (dict(ksc=C.c_void_p(64 * MB + 64)), dict(vsc=C.c_void_p(128 * MB + 64))):
        assert _call(L, True, **kw) == 1


@pytest.mark.parametrize("q8", [False, True])
def test_no_tokens_is_a_no_op(L, q8):
    assert _call(L, q8, T=0, k=NULL, slots=NULL, kp=NULL) == 0


def test_table_refusals(L):
    freq = (C.c_double * 64)(*([1.0] * 64))

    def call(table=FAKE(1), n=10, rot=64, f=freq, factor=1.0):
        return L.pkv_rope_table(table, n, rot, f, factor, NULL)

    bad = (C.c_double * 64)(*([1.0] * 31 + [math.inf] + [1.0] * 32))
    for kw in (dict(n=-1), dict(rot=0), dict(rot=24), dict(rot=144), dict(f=None),
               dict(factor=math.nan), dict(f=bad), dict(table=NULL), dict(table=C.c_void_p(4100))):
        assert call(**kw) == 1, kw
    assert call(n=0, table=NULL) == 0


def test_frequencies():
    import paged_kv_decode_26_gb300 as pkv
    f, m = pkv.rope_frequencies(128)
    assert m == 1.0 and f[0] == 1.0 and f.shape == (64,)
    assert math.isclose(f[63].item(), 10000.0 ** (-126 / 128), rel_tol=1e-14)
    g, m = pkv.rope_frequencies(128, scaling="linear", factor=8.0)
    assert m == 1.0 and torch.allclose(g * 8, f, rtol=1e-14, atol=0)
    g, m = pkv.rope_frequencies(128, scaling="ntk", factor=8.0)
    # the fastest pair as it is, the slowest `factor` times slower
    assert g[0] == 1.0 and math.isclose(g[63].item() * 8, f[63].item(), rel_tol=1e-12)
    g, m = pkv.rope_frequencies(128, scaling="yarn", factor=4.0, original_positions=4096)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40])
    slow = turns < 0.8
    assert torch.allclose(g[slow] * 4, f[slow], rtol=1e-14, atol=0) and slow.any()
    assert ((g <= f * (1 + 1e-14)) & (g >= f / 4 * (1 - 1e-14))).all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=64, base=-1.0),
                dict(rotary_dim=64, factor=0.0), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=2, scaling="ntk", factor=2.0),
                dict(rotary_dim=64, scaling="yarn", factor=2.0),
                dict(rotary_dim=64, base=1.0, scaling="yarn", factor=2.0, original_positions=64)):
        with pytest.raises(ValueError):
            pkv.rope_frequencies(**bad)

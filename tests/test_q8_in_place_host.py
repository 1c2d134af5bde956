"""Outputs of the 8-bit attention that lie on what it reads are refused, the queries
themselves in 16 bits aside.  CPU only: no device is touched."""
import ctypes as C

import pytest

from tests.test_decode_q8_host import FAKE, MB, L, _chunk, _decode  # noqa: F401

POOL = 10 * 16 * 8 * 128


def at(i, offset):
    return C.c_void_p(i * 64 * MB + offset)


@pytest.mark.parametrize("call", [_decode, _chunk])
@pytest.mark.parametrize("kw", [
    dict(out=FAKE(2), od=2), dict(out=at(2, 16)), dict(q=at(1, 16)), dict(out=FAKE(3)),
    dict(out=at(3, POOL - 16)), dict(out=at(4, 4096)), dict(out=FAKE(5)), dict(out=FAKE(6)),
    dict(ks=at(1, 64)), dict(vs=at(1, 4092)),
])
def test_outputs_on_inputs(L, call, kw):  # noqa: F811
    assert call(L, **kw) == 1
    assert L.pkv_last_error_detail()

"""16-bit outputs over long contexts whose values share a sign.  O is summed in
the tensor core, which drops what lies below its accumulator's last bit, always
downwards: at most 2^-23 of O for each 16 keys, added to the bound of
tests/cache_ref.py."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref
from tests.test_long_sums_gpu import _ints, _rows, _same_pages

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
KINDS = [(BF, BF), (FP, FP), (BF, FP)]


def _bound(o, A, d, dtype, out_dtype, once, n):
    return ref.out_bound(o, A, d, dtype, out_dtype, once) + 2.0 ** -23 * (n / 16) * A


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt(D, dtype, out_dtype):
    n = 16000
    q, k, v = _rows(n, D, dtype)
    scale = 0.5 / math.sqrt(D)
    out = torch.empty(n, 2, D, dtype=out_dtype, device="cuda")
    pkv.attn_prompt(out, q.expand(n, 2, D).contiguous().cuda(), k.cuda(), v.cuda(), _ints([0, n]),
                    scale, n)
    for row in (1000, 6001, n - 1):
        o, _, A, d = ref.attend(q[0], k[:row + 1, 0], v[:row + 1, 0], scale)
        ref.check(out[row], o, _bound(o, A, d, dtype, out_dtype, True, row + 1), f"row {row}")


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_weights_decode(D, dtype, out_dtype):
    n, S, scale = 16000, 1200, 0.5 / math.sqrt(D)
    q, k, v, qd, kp, vp, tables, lens = _same_pages(S, n, D, dtype)
    out = torch.empty(S, 2, D, dtype=out_dtype, device="cuda")
    pkv.paged_attn_decode_weights(out, qd, kp, vp, tables, lens, torch.zeros(S, n).cuda(), scale, n)
    o, _, A, d = ref.attend(q[0], k[:, 0], v[:, 0], scale)
    ref.check(out, o.expand(S, 2, D), _bound(o, A, d, dtype, out_dtype, False, n))


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("once", [0, 1])
def test_shared_decode(D, dtype, out_dtype, once):
    n, S, scale = 16000, 304, 0.5 / math.sqrt(D)
    q, k, v, qd, kp, vp, tables, lens = _same_pages(S, n, D, dtype)
    out = torch.empty(S, 2, D, dtype=out_dtype, device="cuda")
    pkv.set_tuning(shared_prefix=once)
    try:
        pkv.paged_attn_decode_shared(out, qd, kp, vp, tables, lens, _ints(list(range(S + 1))),
                                     _ints([n - 32] * S), scale, n, 1, n - 32)
    finally:
        pkv.reset_tuning()
    o, _, A, d = ref.attend(q[0], k[:, 0], v[:, 0], scale)
    ref.check(out, o.expand(S, 2, D), _bound(o, A, d, dtype, out_dtype, True, n))

"""fp32 outputs over long contexts whose values share a sign: every key adds to
the same sums, so an accumulator that drops bits comes out short, more so the
longer the context.  The tolerance is that of tests/cache_ref.py: 2^-17 of
sum p |v| for sums of any length."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def _rows(n, D, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(n, 1, D, generator=g).to(dtype)
    v = (1 + torch.rand(n, 1, D, generator=g)).to(dtype)
    q = torch.randn(1, 2, D, generator=g).to(dtype)
    return q, k, v


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_of_many_keys(D, dtype):
    n = 12000
    q, k, v = _rows(n, D, dtype)
    scale = 0.5 / math.sqrt(D)
    out = torch.empty(n, 2, D, dtype=F32, device="cuda")
    pkv.attn_prompt(out, q.expand(n, 2, D).contiguous().cuda(), k.cuda(), v.cuda(), _ints([0, n]),
                    scale, n)
    for row in (1000, 6001, n - 1):
        o, _, A, d = ref.attend(q[0], k[:row + 1, 0], v[:row + 1, 0], scale)
        ref.check(out[row], o, ref.out_bound(o, A, d, dtype, F32), f"row {row}")


def _same_pages(S, n, D, dtype):
    B = 16
    q, k, v = _rows(n, D, dtype)
    pages = n // B
    tables = torch.arange(pages, dtype=torch.int32, device="cuda").expand(S, -1).contiguous()
    return (q, k, v, q.expand(S, 2, D).contiguous().cuda(), k.view(pages, B, 1, D).cuda(),
            v.view(pages, B, 1, D).cuda(), tables, _ints([n] * S))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_decode_of_long_runs(D, dtype):
    n, S, scale = 16000, 1200, 0.5 / math.sqrt(D)
    q, k, v, qd, kp, vp, tables, lens = _same_pages(S, n, D, dtype)
    out = torch.empty(S, 2, D, dtype=F32, device="cuda")
    w = torch.zeros(S, n, device="cuda")
    pkv.paged_attn_decode_weights(out, qd, kp, vp, tables, lens, w, scale, n)
    o, bound, ws = ref.decode(q, [k], [v], scale, F32)
    ref.check(out, o.expand(S, 2, D), bound, "out")
    some = [0, 1, 599, 1199]
    ref.check(w[some], ws[0][0].expand(4, n), ws[0][1], "weights")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_shared_decode_of_long_prefixes(D, dtype):
    n, S, scale = 16000, 304, 0.5 / math.sqrt(D)
    q, k, v, qd, kp, vp, tables, lens = _same_pages(S, n, D, dtype)
    out = torch.empty(S, 2, D, dtype=F32, device="cuda")
    pkv.paged_attn_decode_shared(out, qd, kp, vp, tables, lens, _ints(list(range(S + 1))),
                                 _ints([n - 32] * S), scale, n, 1, n - 32)
    o, bound, _ = ref.decode(q, [k], [v], scale, F32)
    ref.check(out, o.expand(S, 2, D), bound, "out")

"""Chunks on row tiles whose warps have rows of every kind side by side: none, ones that
see NaN, and ones that look for it over unlike numbers of keys."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref
from tests.cache_ref import check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("H", [1, 2, 8])
@pytest.mark.parametrize("D,B", [(64, 32), (128, 16)])
@pytest.mark.parametrize("m", [1, 5, 17, 33, 100, 131])
def test_ragged_rows_and_nan(m, D, B, H, out_dtype):
    torch.cuda.synchronize()
    pkv.device_errors(clear=True)
    n = 1500
    c = ref.paged([n], B, 1, D, 61)
    g = torch.Generator().manual_seed(62)
    q = torch.randn(m, H, D, generator=g).to(BF)
    scale = 1.0 / math.sqrt(D)
    start = torch.tensor([0, m], dtype=torch.int32).cuda()

    def run():
        out = torch.full((m, H, D), 7.0, dtype=out_dtype, device="cuda")
        pkv.paged_attn_multi_query_q8(out, q.cuda(), start, c["kp"], c["vp"], c["ks"], c["vs"],
                                      c["tables"], c["lens"], scale, m, n)
        return out

    clean = run()
    hidden = torch.ones(m, n, dtype=torch.bool).triu(n - m + 1)
    for h in range(H):
        o, e = ref.attend_bound(q[:, h], c["k"][0][:, 0], c["v"][0][:, 0], scale, out_dtype, hidden,
                                once=out_dtype is not F32, chained=True)
        check(clean[:, h], o, e, f"head {h}")
    nan = torch.zeros(m, H, D, dtype=torch.bool)
    for i, t in enumerate(range(n - m, n, 3)):
        b, d = int(c["tables"][0, t // B]), (37 * i) % D
        c["vp"].view(torch.uint8)[b, t % B, 0, d] = 0x7f
        nan[t - (n - m):, :, d] = True
    out = run()
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    assert torch.equal(out.isnan().cpu(), nan)
    assert torch.equal(out[~nan.cuda()], clean[~nan.cuda()])

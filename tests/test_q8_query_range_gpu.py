"""bf16 queries whose elements lie far apart: what small ones add to a score, exact down
to 2^-31 of the largest and off by 2^-39 of it below."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref
from tests.cache_ref import check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("small", [20, 30, 34, 37, 40])
@pytest.mark.parametrize("bound", [64, 5000])
@pytest.mark.parametrize("chunk", [False, True])
def test_small_elements(small, bound, chunk):
    torch.cuda.synchronize()
    pkv.device_errors(clear=True)
    H, D, B, n = 4, 64, 16, 64
    c = ref.paged([n], B, 1, D, 111)
    g = torch.Generator().manual_seed(112)
    q = torch.zeros(1, H, D)
    q[..., 0] = 1.5                                # meets keys of zero
    q[..., 1:] = (torch.randn(1, H, D - 1, generator=g).sign() *
                  (torch.rand(1, H, D - 1, generator=g) + 1.0)) * 2.0 ** -small
    q = (q * 2.0 ** 40).to(BF)
    k8 = c["kp"].view(torch.uint8)
    for j in range(n // B):
        b = int(c["tables"][0, j])
        k8[b, :, 0, 0] = 0
    c["k"][0][:, 0, 0] = 0.0
    # scores of a few units, by the small elements alone
    scale = 2.0 ** (small - 40) / math.sqrt(D)
    out = torch.full(q.shape, math.nan, device="cuda")
    rest = (c["kp"], c["vp"], c["ks"], c["vs"], c["tables"], c["lens"], scale)
    if chunk:
        start = torch.tensor([0, 1], dtype=torch.int32).cuda()
        pkv.paged_attn_multi_query_q8(out, q.cuda(), start, *rest, 1, bound)
    else:
        pkv.paged_attn_decode_q8(out, q.cuda(), *rest, bound)
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    k, v = c["k"][0][:, 0], c["v"][0][:, 0]
    top = q.double().abs().max()
    for h in range(H):
        o, e = ref.attend_bound(q[:, h], k, v, scale, F32, chained=True)
        # an element off by 2^-39 of the largest: a score by that times |k|, a weight by
        # twice its exponential's change
        off = 0.0 if small <= 30 else 2 * scale * 2.0 ** -39 * top * k.abs().sum(-1).max()
        p = torch.softmax(q[:, h].double() @ k.T * scale, -1)
        check(out[:, h], o, e + off * math.exp(off) * (p @ v.abs()), f"head {h}")

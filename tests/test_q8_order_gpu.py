"""Chunks over 8-bit pages on both sides of the bounds from which CTAs take the longest
contexts first, against the plain form."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref
from tests.cache_ref import check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("S,H,Hk,D,B", [(3, 8, 2, 128, 16), (80, 2, 1, 64, 16), (100, 4, 4, 64, 32)])
def test_both_orders(S, H, Hk, D, B):
    torch.cuda.synchronize()
    pkv.device_errors(clear=True)
    g = torch.Generator().manual_seed(91)
    seqs = [(int(torch.randint(0, 40, (1,), generator=g)), int(torch.randint(40, 300, (1,), generator=g)))
            for _ in range(S)]
    seqs[S // 2], seqs[-1] = (70, 1200), (33, 2500)
    c = ref.paged([n for _, n in seqs], B, Hk, D, 92)
    starts = [0]
    for m, _ in seqs:
        starts.append(starts[-1] + m)
    q = torch.randn(starts[-1], H, D, generator=g).to(BF)
    want, bound = (torch.zeros(starts[-1], H, D, dtype=torch.float64) for _ in range(2))
    scale = 1.0 / math.sqrt(D)
    for s, (m, n) in enumerate(seqs):
        hidden = torch.ones(m, n, dtype=torch.bool).triu(n - m + 1)
        for h in range(H if m else 0):
            rows = slice(starts[s], starts[s + 1])
            want[rows, h], bound[rows, h] = ref.attend_bound(
                q[rows, h], c["k"][s][:, h // (H // Hk)], c["v"][s][:, h // (H // Hk)], scale, F32,
                hidden, chained=True)
    start = torch.tensor(starts, dtype=torch.int32).cuda()
    # (chunks of more than half the context count as prompts)
    for max_q, max_len in ((70, 2559), (70, 2560), (70, 3199), (70, 3200), (1281, 2560), (70, 8192),
                           (5000, 8191), (5000, 8192)):
        out = torch.full((starts[-1], H, D), math.nan, device="cuda")
        pkv.paged_attn_multi_query_q8(out, q.cuda(), start, c["kp"], c["vp"], c["ks"], c["vs"],
                                      c["tables"], c["lens"], scale, max_q, max_len)
        torch.cuda.synchronize()
        assert pkv.device_errors(clear=True) == 0
        check(out, want, bound, f"bounds {max_q}, {max_len}")

"""8-bit attention that writes over its queries: the same bits as apart from them."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,B,H,Hk", [(64, 16, 8, 8), (128, 32, 16, 2), (128, 16, 4, 4)])
@pytest.mark.parametrize("bound", [700, 40000])
def test_decode(D, B, H, Hk, dtype, bound):
    """Whole contexts and pieces."""
    _clean()
    lens = [0, 1, 17, 700, 33, 512] * 4
    c = ref.paged(lens, B, Hk, D, 101)
    q = torch.randn(len(lens), H, D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    args = (c["kp"], c["vp"], c["ks"], c["vs"], c["tables"], c["lens"], 1 / math.sqrt(D), bound)
    want = pkv.paged_attn_decode_q8(torch.empty_like(q), q, *args)
    for _ in range(5):
        x = q.clone()
        pkv.paged_attn_decode_q8(x, x, *args)
        assert torch.equal(x, want)
    assert _clean() == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("seqs,D,B,H,Hk,bound", [
    ([(3, 40), (8, 300), (0, 5), (5, 5)], 64, 16, 8, 4, 300),           # tokens by themselves
    ([(70, 700), (9, 2000), (300, 300)], 128, 16, 8, 2, 2000),          # row tiles, keys in parts
    ([(130, 300)] * 20, 64, 32, 16, 16, 300),                           # whole items
])
def test_chunks(seqs, D, B, H, Hk, bound, dtype):
    _clean()
    c = ref.paged([n for _, n in seqs], B, Hk, D, 102)
    starts = [0]
    for m, _ in seqs:
        starts.append(starts[-1] + m)
    q = torch.randn(starts[-1], H, D, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    start = torch.tensor(starts, dtype=torch.int32).cuda()
    args = (c["kp"], c["vp"], c["ks"], c["vs"], c["tables"], c["lens"], 1 / math.sqrt(D),
            max(m for m, _ in seqs), bound)
    want = pkv.paged_attn_multi_query_q8(torch.empty_like(q), q, start, *args)
    for _ in range(5):
        x = q.clone()
        pkv.paged_attn_multi_query_q8(x, x, start, *args)
        assert torch.equal(x, want)
    assert _clean() == 0

"""Prompts whose last rows fill warps in part, with NaN in the last values: rows of one
warp look for it over unlike numbers of keys, or not at all."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,Hk,D", [(8, 1, 128), (4, 4, 128), (2, 1, 64)])
@pytest.mark.parametrize("lens", [[1, 5, 33], [131, 17, 300], [257]])
def test_ragged_prompts_and_nan(lens, H, Hk, D, dtype):
    torch.cuda.synchronize()
    pkv.device_errors(clear=True)
    g = torch.Generator().manual_seed(71)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    T = starts[-1]
    q, k, v = (torch.randn(T, h, D, generator=g).to(dtype).cuda() for h in (H, Hk, Hk))
    start = torch.tensor(starts, dtype=torch.int32).cuda()

    def run():
        out = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
        pkv.attn_prompt(out, q, k, v, start, 1.0 / math.sqrt(D), max(lens))
        return out

    clean = run()
    assert not clean.isnan().any()
    nan = torch.zeros(T, H, D, dtype=torch.bool)
    G = H // Hk
    for a, b in zip(starts, starts[1:]):
        for i, t in enumerate(range(max(a, b - 40), b, 3)):
            d, kvh = (29 * i) % D, i % Hk
            v[t, kvh, d] = math.nan
            nan[t:b, kvh * G:(kvh + 1) * G, d] = True
    out = run()
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    assert torch.equal(out.isnan().cpu(), nan)
    assert torch.equal(out[~nan.cuda()], clean[~nan.cuda()])

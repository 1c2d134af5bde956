"""The serving loop of the cache operators with its shared steps' prefix attended
once for the group, and by every member alone, whatever the automatic choice
would be for so short a prefix."""
import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests.test_cache_loop_gpu import test_serving_loop as serving_loop

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("once", [0, 1])
@pytest.mark.parametrize("H,Hk,D,B,dtype", [(8, 2, 128, 16, torch.bfloat16),
                                            (4, 4, 64, 32, torch.float16)])
def test_both_ways(once, H, Hk, D, B, dtype):
    pkv.set_tuning(shared_prefix=once)
    try:
        serving_loop(H, Hk, D, B, dtype)
    finally:
        pkv.reset_tuning()

"""paged_attn_decode_shared with its prefixes attended once gives the ordinary
decode's result to the ordinary decode's tolerance, 16-bit outputs included:
softmax weights in two 16-bit parts (tests/cache_ref.py), whatever the automatic
choice does.  fp16 outputs below 2^-14 have steps of 2^-24: 2^-25 is added."""
import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref
from tests import test_decode_shared_gpu as base

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("out_dtype", [BF, FP])
@pytest.mark.parametrize("lens,starts,prefix,H,Hk,D,B,dtype,_", base.CASES)
def test_decodes_tolerance(lens, starts, prefix, H, Hk, D, B, dtype, _, out_dtype):
    base._clean()
    c = base._problem(lens, starts, prefix, H, Hk, D, B, dtype)
    pkv.set_tuning(shared_prefix=1)
    try:
        out = base._run(c, starts, prefix, out_dtype, max(lens))
    finally:
        pkv.reset_tuning()
    assert base._clean() == 0
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], out_dtype)
    ref.check(out, o, bound + (2.0 ** -25 if out_dtype == FP else 0.0))

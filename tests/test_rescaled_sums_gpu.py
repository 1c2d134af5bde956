"""The schedule of 16-bit outputs where rows have to be rescaled: scales that are
zero, negative or large, and scores that grow from key tile to key tile, so that
a row's reference moves and O is multiplied in tensor memory.  Prompts and
prefixes attended once, every output type, both head sizes, with and without
grouped heads, against the 64-bit form (tolerances: tests/cache_ref.py).  That
file's rounding of the output is relative to the value; fp16 below 2^-14 has steps
of 2^-24 whatever the value, so a rounding there is off by up to 2^-25 (an output
of 1.5e-6 by 2.7e-8, 0.91 of that): added for fp16 outputs."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref
from tests.test_large_scores_gpu import _pages

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
KINDS = [(BF, BF), (BF, FP), (BF, F32), (FP, FP), (FP, BF), (FP, F32)]
HEADS = [(2, 2, 64), (8, 1, 64), (4, 4, 128), (8, 2, 128)]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(rows, n, H, Hk, D, dtype, growth, seed=3):
    """q [rows, H, D], k, v [n, Hk, D]; with growth, scores of
    key t are about (1 + growth t) times as large as those of key 0, some rows'
    positive and some negative (their maximum stays at the first tile)."""
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(m, h, D, generator=g) for m, h in ((rows, H), (n, Hk), (n, Hk)))
    if growth:
        q = q.abs() * (1 - 2 * (torch.arange(rows) % 5 == 4).float())[:, None, None]
        k = k.abs() * (1 + growth * torch.arange(n))[:, None, None]
    return q.to(dtype), k.to(dtype), v.to(dtype)


def _check(out, o, bound, what=""):
    ref.check(out, o, bound + (2.0 ** -25 if out.dtype == FP else 0.0), what)


def _prompt(q, k, v, scale, out_dtype):
    n, H, D = q.shape
    G = H // k.shape[1]
    out = torch.full((n, H, D), float("nan"), dtype=out_dtype, device="cuda")
    pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(), _ints([0, n]), scale, n)
    hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
    for h in range(H):
        o, _, A, d = ref.attend(q[:, h], k[:, h // G], v[:, h // G], scale, hidden)
        _check(out[:, h], o, ref.out_bound(o, A, d, q.dtype, out_dtype, out_dtype != F32),
               f"head {h}")


def _shared(q, k, v, scale, out_dtype, lens, prefix):
    S, H, D = q.shape
    kp, vp, tables, ln = _pages(lens, 16, k, v)
    out = torch.full((S, H, D), float("nan"), dtype=out_dtype, device="cuda")
    pkv.set_tuning(shared_prefix=1)
    try:
        pkv.paged_attn_decode_shared(out, q.cuda(), kp, vp, tables, ln, _ints([0, S]),
                                     _ints([prefix]), scale, max(lens), S, prefix)
    finally:
        pkv.reset_tuning()
    o, bound, _ = ref.decode(q, [k[:n] for n in lens], [v[:n] for n in lens], scale, out_dtype,
                             once=out_dtype != F32)
    _check(out, o, bound)


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_prompt_scales(scale, H, Hk, D, dtype, out_dtype):
    _prompt(*_rows(400, 400, H, Hk, D, dtype, 0), scale, out_dtype)


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("scale", [0.5, -0.5])
def test_prompt_growing_scores(scale, H, Hk, D, dtype, out_dtype):
    _prompt(*_rows(700, 700, H, Hk, D, dtype, 1 / 60), scale / math.sqrt(D), out_dtype)


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("H,Hk,D", HEADS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_prefix_scales(scale, H, Hk, D, dtype, out_dtype):
    lens = [330, 300, 400, 380, 320]
    _shared(*_rows(5, 400, H, Hk, D, dtype, 0), scale, out_dtype, lens, 320)


# (so many kv heads that the prefix's splits are 3 to 7 key tiles long)
@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("H,Hk,D", [(32, 32, 64), (64, 16, 64), (32, 32, 128), (64, 16, 128)])
@pytest.mark.parametrize("scale", [0.5, -0.5])
def test_prefix_growing_scores(scale, H, Hk, D, dtype, out_dtype):
    lens = [4100, 4096, 4200] * 4
    _shared(*_rows(len(lens), 4200, H, Hk, D, dtype, 1 / 60), scale / math.sqrt(D), out_dtype,
            lens, 4096)

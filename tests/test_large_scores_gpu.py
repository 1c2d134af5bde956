"""Scores far beyond what a softmax resolves -- 2^14 to 2^100 in units of its
base-2 exponent, from finite 16-bit inputs -- in every operator that attends.

One key leads every other by 2^-7 of the score's size or more, so by hundreds of
units, and every other weight is 0 in fp32 as in 64 bits: a row of the output
is the leading key's row of V.  The products are exact (powers of two times 6-bit
numbers), the scale is not, so a scaled score of 2^27 is off by several units in
fp32: a weight formed from an unrounded product and a rounded maximum, or from a
reference that fp32 cannot hold, then leaves the range of fp16, or that of fp32.

Tolerances: tests/cache_ref.py with one weight of 1 (d = 0: the leading weight
and the sum that divides it are the same number)."""

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
# (type of q, k and v, type of the output, log2 of the scores)
SIZES = ([(FP, o, x) for o in (FP, F32) for x in (14, 16, 20, 24, 27, 30, 34, 38)]
         + [(BF, o, x) for o in (BF, F32) for x in (14, 16, 20, 27, 30, 34, 37, 40, 100)])
# where a new key takes the lead: in the first rows, at the ends of chunks and tiles
LEADS = (0, 1, 5, 16, 40, 127, 128, 129, 200, 311, 512, 640)


def _factors(n, below):
    """Scores of n keys in units of 2^size: from 1 up, or (below) from -2 up."""
    m = torch.zeros(n)
    lead = 0
    for t in range(n):
        if t in LEADS:
            lead += 2
        m[t] = lead if t in LEADS else t % 2
    return (m / 64 - 2) if below else (m / 64 + 1)


def _leading(n):
    """The leading key among the first i + 1, for each i."""
    return torch.tensor([max(t for t in LEADS if t <= i) for i in range(n)])


def _rows(n, rows, H, Hk, D, dtype, size, below, flip):
    """q [rows, H, D], k, v [n, Hk, D], scale.  Rows of several sizes, from
    2^size down to 2^14, lie next to each other."""
    g = torch.Generator().manual_seed(size + D)
    big = 14 if dtype == FP else max(14, size // 3)
    sign = 1 - 2 * torch.randint(2, (D,), generator=g).float()
    down = torch.tensor([0, size - max(14, size - 6), size - 14, 0])
    q = (sign * 2.0 ** big).expand(rows, H, D) * 2.0 ** -down[torch.arange(rows) % 4].float()[
        :, None, None]
    k = (sign * 2.0 ** big) * _factors(n, below)[:, None, None].expand(n, Hk, D)
    v = torch.randn(n, Hk, D, generator=g)
    scale = 0.7 * 2.0 ** (size - 2 * big) / D
    if flip:
        k, scale = -k, -scale
    return q.to(dtype).contiguous(), k.to(dtype).contiguous(), v.to(dtype), scale


def _check(out, want, dtype, once, what):
    """out, want [R, D]"""
    want = want.double()
    b = ref.out_bound(want, want.abs(), torch.zeros(want.shape[0]), dtype, out.dtype, once)
    ref.check(out, want, b, what)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype,size", SIZES)
def test_prompt(dtype, out_dtype, size, D):
    n, H, Hk = 700, 4, 2
    lead = _leading(n)
    for below, flip in ((False, False), (True, False), (False, True)):
        q, k, v, scale = _rows(n, n, H, Hk, D, dtype, size, below, flip)
        out = torch.empty(n, H, D, dtype=out_dtype, device="cuda")
        pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(),
                        torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale, n)
        for h in range(H):
            _check(out[:, h], v[lead, h // 2], dtype, out_dtype != F32, f"head {h}")


def _pages(lens, B, k, v):
    """Every sequence at the same pages, rows behind the longest are NaN."""
    n = max(lens)
    pages = (n + B - 1) // B
    pools = []
    for x in (k, v):
        pool = torch.full((pages * B, *x.shape[1:]), float("nan"), dtype=x.dtype)
        pool[:n] = x[:n]
        pools.append(pool.view(pages, B, *x.shape[1:]).cuda())
    tables = torch.arange(pages, dtype=torch.int32, device="cuda").expand(len(lens), -1)
    return (*pools, tables.contiguous(), torch.tensor(lens, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype,size", SIZES)
@pytest.mark.parametrize("S", [5, 700])
def test_weights_decode(dtype, out_dtype, size, D, S):
    """S = 5: sequences cut into pieces; 700: runs of whole sequences."""
    lens = ([700, 1, 130, 650, 17] * (S // 5))
    H, Hk, n = 4, 2, 700
    at = _leading(n)[torch.tensor(lens) - 1]
    for below, flip in ((False, False), (True, False), (False, True)):
        q, k, v, scale = _rows(n, S, H, Hk, D, dtype, size, below, flip)
        kp, vp, tables, ln = _pages(lens, 16, k, v)
        out = torch.empty(S, H, D, dtype=out_dtype, device="cuda")
        w = torch.zeros(S, n, device="cuda")
        pkv.paged_attn_decode_weights(out, q.cuda(), kp, vp, tables, ln, w, scale, n)
        for h in range(H):
            _check(out[:, h], v[at, h // 2], dtype, False, f"head {h}")
        want = torch.zeros(S, n, dtype=torch.float64)
        want[torch.arange(S), at] = H
        ref.check(w, want, want * (2.0 ** -18 + H * 2.0 ** -24) + 1e-30, "weights")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype,size", SIZES)
@pytest.mark.parametrize("once", [0, 1])
def test_shared_decode(dtype, out_dtype, size, D, once):
    lens = [700, 512, 650, 515, 700, 528, 640]
    S, H, Hk, n, prefix = len(lens), 4, 2, 700, 512
    at = _leading(n)[torch.tensor(lens) - 1]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pkv.set_tuning(shared_prefix=once)
    try:
        for below, flip in ((False, False), (True, False), (False, True)):
            q, k, v, scale = _rows(n, S, H, Hk, D, dtype, size, below, flip)
            kp, vp, tables, ln = _pages(lens, 16, k, v)
            out = torch.empty(S, H, D, dtype=out_dtype, device="cuda")
            pkv.paged_attn_decode_shared(out, q.cuda(), kp, vp, tables, ln, ints([0, S]),
                                         ints([prefix]), scale, n, S, prefix)
            for h in range(H):
                _check(out[:, h], v[at, h // 2], dtype, out_dtype != F32, f"head {h}")
    finally:
        pkv.reset_tuning()
    assert pkv.device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype,out_dtype", [(BF, FP), (FP, FP), (BF, F32)])
def test_prompts_do_not_change_with_their_neighbours(dtype, out_dtype):
    """The rows behind a sequence's last ones in a tile are the next sequence's:
    its size of scores is not this one's, bit for bit (of some hundred thousand
    elements, so that a difference of roundings would show)."""
    n, S = 71, 80
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(n * S, h, 128, generator=g).to(dtype) for h in (8, 2, 2))
    odd = (torch.arange(n * S) // n % 2 == 1)[:, None, None]
    starts = torch.arange(0, n * S + 1, n, dtype=torch.int32, device="cuda")
    got = []
    for big in (1.0, 2.0 ** 12, float("inf")):
        q2 = torch.where(odd, q * big, q)
        out = torch.empty(n * S, 8, 128, dtype=out_dtype, device="cuda")
        pkv.attn_prompt(out, q2.cuda(), k.cuda(), v.cuda(), starts, 3.0, n)
        got.append(out[~odd[:, 0, 0].cuda()].clone())
    assert torch.isfinite(got[0]).all()
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])

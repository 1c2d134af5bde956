"""attn_prompt against a plain 64-bit form (tests/cache_ref.py, where the
tolerances are derived; the softmax weights are rounded once for 16-bit
outputs)."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from paged_kv_decode_26_gb300 import _lib
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


def _starts(lens, lead=0):
    s = [lead]
    for n in lens:
        s.append(s[-1] + n)
    return s


def _inputs(T, H, Hk, D, dtype, fused=False, seed=1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, H + 2 * Hk, D, generator=g) * scale).to(dtype)
    parts = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    if fused:
        dev = qkv.cuda()
        return parts, (dev[:, :H], dev[:, H:H + Hk], dev[:, H + Hk:])
    return parts, tuple(p.contiguous().cuda() for p in parts)


def _reference(parts, starts, scale, out_dtype, heads=None):
    """(out, bound) of the listed heads, [T, len(heads), D]."""
    q, k, v = parts
    T, H, D = q.shape
    G = H // k.shape[1]
    heads = range(H) if heads is None else heads
    out = torch.zeros(T, len(heads), D, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for a, b in zip(starts, starts[1:]):
        n = b - a
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        for i, h in enumerate(heads):
            if n == 0:
                continue
            o, _, A, d = ref.attend(q[a:b, h], k[a:b, h // G], v[a:b, h // G], scale, hidden)
            out[a:b, i] = o
            bound[a:b, i] = ref.out_bound(o, A, d, q.dtype, out_dtype, once=out_dtype != F32)
    return out, bound


CASES = [
    # lens, H, Hk, D, dtype, out, fused
    ([1], 1, 1, 64, FP, FP, False),
    ([1], 8, 1, 128, BF, F32, False),
    ([0, 3, 0, 127, 0], 4, 2, 128, BF, BF, True),
    ([128, 129, 255, 256, 257], 2, 2, 64, BF, BF, True),
    ([5, 200, 33, 1, 64], 8, 2, 128, FP, F32, True),
    ([31, 32, 33, 63, 64, 65, 66], 8, 1, 64, BF, BF, False),
    ([700], 4, 4, 128, BF, BF, False),
    ([513, 1, 1025], 8, 1, 128, BF, BF, True),
    ([1, 2, 3, 4, 5, 6, 7, 8] * 25, 6, 3, 64, FP, FP, False),
    ([300] * 12, 16, 8, 128, BF, F32, False),
    ([2100, 77], 2, 1, 64, BF, BF, True),
]


@pytest.mark.parametrize("lens,H,Hk,D,dtype,out_dtype,fused", CASES)
def test_prompt(lens, H, Hk, D, dtype, out_dtype, fused):
    _clean()
    starts = _starts(lens)
    T = starts[-1]
    parts, dev = _inputs(T, H, Hk, D, dtype, fused)
    out = torch.full((T, H, D), float("nan"), dtype=out_dtype, device="cuda")
    scale = 1 / math.sqrt(D)
    pkv.attn_prompt(out, *dev, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale,
                    max(lens))
    assert _clean() == 0
    ref.check(out, *_reference(parts, starts, scale, out_dtype))


@pytest.mark.parametrize("H,Hk,D,n,dtype", [(32, 8, 128, 4500, BF), (8, 8, 64, 3500, FP)])
def test_long_prompt_some_heads(H, Hk, D, n, dtype):
    _clean()
    starts = _starts([n, 600, n // 3])
    parts, dev = _inputs(starts[-1], H, Hk, D, dtype, True)
    out = torch.empty(starts[-1], H, D, dtype=dtype, device="cuda")
    pkv.attn_prompt(out, *dev, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                    1 / math.sqrt(D), n)
    assert _clean() == 0
    heads = [0, H // 2 + 1, H - 1]
    o, b = _reference(parts, starts, 1 / math.sqrt(D), dtype, heads)
    ref.check(out[:, heads], o, b)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_prompt_scales(scale):
    starts = _starts([150, 40])
    parts, dev = _inputs(190, 4, 2, 64, BF)
    out = torch.empty(190, 4, 64, dtype=F32, device="cuda")
    pkv.attn_prompt(out, *dev, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale, 150)
    ref.check(out, *_reference(parts, starts, scale, F32), f"scale {scale}")


def test_prompt_growing_scores():
    """Rows whose maximum grows from tile to tile: O is rescaled."""
    n, D = 900, 64
    parts, _ = _inputs(n, 2, 1, D, BF)
    q, k, v = [x.clone() for x in parts]
    k *= (1 + torch.arange(n)[:, None, None] / 60.0)
    q = (q.abs() * 2).to(BF)
    k = (k.abs()).to(BF)
    out = torch.empty(n, 2, D, dtype=F32, device="cuda")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(), starts, 0.125, n)
    ref.check(out, *_reference((q, k, v), [0, n], 0.125, F32))


def test_rows_of_no_sequence_stay_and_neighbours_do_not_leak():
    """Tokens before the first and behind the last sequence are neither read
    into a result nor written; a poisoned neighbour stays by itself."""
    _clean()
    lens, lead, tail = [70, 50, 200], 9, 40
    starts = _starts(lens, lead)
    T = starts[-1] + tail
    parts, _ = _inputs(T, 4, 2, 128, BF)
    q, k, v = [x.clone() for x in parts]
    bad = [slice(0, lead), slice(starts[1], starts[2]), slice(starts[-1], T)]
    for s in bad:
        k[s] = float("nan")
        v[s] = float("inf")
        q[s] = float("nan")
    out = torch.full((T, 4, 128), 7.0, dtype=BF, device="cuda")
    pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(),
                    torch.tensor(starts, dtype=torch.int32, device="cuda"), 0.1, 200)
    assert _clean() == 0
    o, b = _reference(parts, starts, 0.1, BF)
    for i in (0, 2):
        a, e = starts[i], starts[i + 1]
        ref.check(out[a:e], o[a:e], b[a:e])
    assert (out[:lead] == 7).all() and (out[starts[-1]:] == 7).all()


@pytest.mark.parametrize("H,Hk,D,dtype,out_dtype", [(4, 2, 128, BF, BF), (8, 1, 64, FP, F32),
                                                    (2, 2, 128, FP, FP)])
def test_nan_and_infinities_reach_only_the_queries_that_see_them(H, Hk, D, dtype, out_dtype):
    """V rows with NaN and infinities: hidden from earlier tokens, they leave
    no trace there.  Tokens that see them get no number in those columns: NaN,
    or the infinity -- a weight enters the product as a rounded number, or as
    the sum of two of which the second may be 0 or negative, and infinity times
    0, or infinity minus infinity, is NaN."""
    _clean()
    lens = [300, 150, 40]
    starts = _starts(lens)
    parts, _ = _inputs(starts[-1], H, Hk, D, dtype)
    q, k, v = [x.clone() for x in parts]
    inf, nan = float("inf"), float("nan")
    v[170, 0, 3] = nan
    v[255, 0, 5] = inf
    v[299, Hk - 1, 7] = -inf
    v[starts[1] + 149, 0, 1] = nan                 # the last token of a sequence
    v[starts[2], Hk - 1, 9] = inf                  # the first one
    v[starts[2] + 20, Hk - 1, 9] = -inf            # and the opposite: NaN from here
    k[starts[1] + 100, 0, 2] = nan                 # a key: NaN from its token on
    out = torch.empty(starts[-1], H, D, dtype=out_dtype, device="cuda")
    scale = 1 / math.sqrt(D)
    pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(),
                    torch.tensor(starts, dtype=torch.int32, device="cuda"), scale, 300)
    assert _clean() == 0
    got = out.double().cpu()
    ok = lambda x: torch.nan_to_num(x.double(), nan=0.0, posinf=0.0, neginf=0.0).to(dtype)  # noqa
    want, bound = _reference((q, ok(k), ok(v)), starts, scale, out_dtype)
    for a, b in zip(starts, starts[1:]):
        for i in range(a, b):
            for h in range(H):
                g = h // (H // Hk)
                if torch.isnan(k[a:i + 1, g]).any():
                    assert torch.isnan(got[i, h]).all()
                    continue
                add = torch.where(torch.isfinite(v[a:i + 1, g]), 0.0, v[a:i + 1, g].double()).sum(0)
                strange = ~torch.isfinite(add)
                assert torch.equal(~torch.isfinite(got[i, h]), strange), (i, h)
                assert torch.isnan(got[i, h][torch.isnan(add)]).all(), (i, h)
                err = (got[i, h] - want[i, h]).abs()[~strange]
                assert (err <= bound[i, h][~strange]).all(), (i, h)


def test_prompt_flags_bad_bounds():
    _clean()
    _, dev = _inputs(100, 2, 2, 64, BF)
    out = torch.full((100, 2, 64), 7.0, dtype=BF, device="cuda")
    for starts, max_len in (([0, 50, 40, 60], 60), ([0, 60, 101], 60), ([-1, 20], 60),
                            ([0, 61], 60)):
        pkv.attn_prompt(out, *dev, torch.tensor(starts, dtype=torch.int32, device="cuda"), 0.1,
                        max_len)
        assert _clean() == _lib.DEVERR_CONTEXT, starts


def test_prompt_repeats_and_graph_and_stream():
    starts = torch.tensor(_starts([300, 80]), dtype=torch.int32, device="cuda")
    _, dev = _inputs(380, 8, 2, 128, BF)
    out = torch.empty(380, 8, 128, dtype=BF, device="cuda")
    pkv.attn_prompt(out, *dev, starts, 0.09, 300)
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.attn_prompt(out, *dev, starts, 0.09, 300)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.attn_prompt(out, *dev, starts, 0.09, 300, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("H,Hk,out_dtype", [(8, 8, BF), (16, 8, F32)])
def test_long_prompts_beyond_the_cache(H, Hk, out_dtype):
    """Long prompts whose K and V exceed L2 (items of a head go together), of
    ragged lengths: sampled rows of every sequence and head."""
    _clean()
    lens, D = [9000, 4097, 1, 0, 700, 8192, 5000, 6001], 128
    starts = _starts(lens, lead=3)
    parts, dev = _inputs(starts[-1] + 5, H, Hk, D, BF, True)
    out = torch.full((starts[-1] + 5, H, D), 7.0, dtype=out_dtype, device="cuda")
    scale = 1 / math.sqrt(D)
    pkv.attn_prompt(out, *dev, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale, 9000)
    assert _clean() == 0
    assert (out[:3] == 7).all() and (out[-5:] == 7).all()
    q, k, v = parts
    g = torch.Generator().manual_seed(2)
    for a, n in zip(starts, lens):
        if n == 0:
            continue
        rows = torch.unique(torch.cat([torch.tensor([0, n - 1, n // 2]),
                                       torch.randint(n, (12,), generator=g)]))
        hidden = torch.arange(n)[None] > rows[:, None]
        for h in range(H):
            o, _, A, d = ref.attend(q[a + rows, h], k[a:a + n, h * Hk // H],
                                    v[a:a + n, h * Hk // H], scale, hidden)
            b = ref.out_bound(o, A, d, BF, out_dtype, once=out_dtype != F32)
            ref.check(out[a + rows, h], o, b, f"sequence at {a}, head {h}")


def test_bounds_that_allow_more_than_2_to_31_tiles():
    """A hundred thousand sequences, nearly all empty, under a bound of a
    million tokens each: several launches, each passing over empty items."""
    _clean()
    S, T, H, D = 100000, 1 << 20, 8, 64
    lens = torch.zeros(S, dtype=torch.int64)
    lens[0], lens[50000], lens[S - 1] = 100, 333, 1
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, H, D, generator=g, device="cuda").to(BF)
    k, v = (torch.randn(T, 1, D, generator=g, device="cuda").to(BF) for _ in range(2))
    out = torch.full((T, H, D), 7.0, dtype=BF, device="cuda")
    pkv.attn_prompt(out, q, k, v, starts.int().cuda(), 0.125, T)
    assert _clean() == 0
    n = int(starts[-1])
    assert (out[n:] == 7).all()
    real = [0, 100, 433, 434]
    o, b = _reference(tuple(x[:n].cpu() for x in (q, k, v)), real, 0.125, BF)
    ref.check(out[:n], o, b)

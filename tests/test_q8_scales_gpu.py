"""8-bit attention with value scales from one end of the range to the other, against
the plain 64-bit form: contexts of one size, blocks of far smaller and larger values
beside ordinary ones, and blocks of hardly any value that softmax weighs most."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref
from tests.cache_ref import check

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
# fp32's least normal number: what is smaller may count as 0, in a product with a scale,
# and in an output
LEAST = 2.0 ** -126


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


def _problem(seqs, H, Hk, D, B, dtype, exponents, seed, gap=None):
    """seqs (new tokens, context); block j of a sequence has values of scale
    2^exponents[j % ..] (None: near 1/200; "zero": the least, and codes of 0).  gap: the
    keys of blocks below 2^-60 point along one direction, of every query too, and
    score that much (in powers of two) above the others, at a scale of 1 / sqrt(D)."""
    c = ref.paged([n for _, n in seqs], B, Hk, D, seed)
    g = torch.Generator().manual_seed(seed + 50)
    T = sum(m for m, _ in seqs)
    q = torch.randn(T, H, D, generator=g)
    if gap is not None:
        q[..., 0] = 4.0
    c["q"] = q.to(dtype)
    c["starts"] = [0]
    for s, (m, n) in enumerate(seqs):
        c["starts"].append(c["starts"][-1] + m)
        for j in range(-(-n // B)):
            e = exponents[j % len(exponents)]
            if e is None:
                continue
            b, rows = int(c["tables"][s, j]), slice(j * B, min(n, j * B + B))
            new = 2.0 ** (-117 if e == "zero" else e)
            if e == "zero":
                c["vp"].view(torch.uint8)[b] = 0
                c["v"][s][rows] = 0.0
            else:
                c["v"][s][rows] *= new / c["vs"][b].cpu().double()[:, None]
            c["vs"][b] = new
            if gap is not None and (e == "zero" or e < -60):
                unit = torch.zeros(Hk, D, dtype=torch.float64)
                unit[:, 0] = 256.0
                up = gap * math.log(2.0) * math.sqrt(D) / (4.0 * 256.0)
                c["ks"][b] = up
                up = float(c["ks"][b, 0])
                c["kp"].view(torch.uint8)[b, :rows.stop - rows.start] = \
                    unit.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
                c["k"][s][rows] = unit * up
    c["q_start"] = torch.tensor(c["starts"], dtype=torch.int32).cuda()
    return c


def _want(c, scale, out_dtype, once):
    q = c["q"]
    T, H, D = q.shape
    out, bound = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    for s, (a, b) in enumerate(zip(c["starts"], c["starts"][1:])):
        k, v = c["k"][s], c["v"][s]
        n, G = k.shape[0], H // k.shape[1]
        hidden = torch.ones(b - a, n, dtype=torch.bool).triu(n - (b - a) + 1)
        for h in range(H):
            o, e = ref.attend_bound(q[a:b, h], k[:, h // G], v[:, h // G], scale, out_dtype, hidden,
                                    once=once, chained=True)
            # (the form's floor of 1e-30 is above these values: fp32's instead, of
            # each of the values and of the result)
            out[a:b, h], bound[a:b, h] = o, e - 1e-30 + 500 * LEAST
    return out, bound


EXPONENTS = [
    [-117], [-101], [-104, -117], [-122], [112],        # contexts of one size
    [None, -117], [-117, None], [None, -101, None],     # beside ordinary ones
    ["zero", None], [None, "zero", "zero"],
    [-117, 100, None, -60, -61, 17], ["zero", 110, -117], [90, None, "zero", -40],
]
GAPS = [([None, -117], 12.0), ([None, -100, None], 60.0), (["zero", None], 12.0),
        ([None, "zero"], 50.0), ([None, "zero"], 90.0), ([110, "zero", None], 30.0),
        ([110, "zero"], 100.0), ([None, -117], 118.0), (["zero", 30, -117], 120.0)]
ALL = [(e, None) for e in EXPONENTS] + GAPS


@pytest.mark.parametrize("D,B,out_dtype", [(64, 16, F32), (128, 32, BF), (128, 16, F32)])
@pytest.mark.parametrize("exponents,gap", ALL)
@pytest.mark.parametrize("bound", [700, 20000])
def test_decode(D, B, out_dtype, exponents, gap, bound):
    """Whole contexts, and pieces."""
    _clean()
    c = _problem([(1, n) for n in (1, B + 3, 100, 700)], 8, 2, D, B, BF, exponents, 31, gap)
    out = torch.full(c["q"].shape, math.nan, dtype=out_dtype, device="cuda")
    scale = 1.0 / math.sqrt(D)
    pkv.paged_attn_decode_q8(out, c["q"].cuda(), c["kp"], c["vp"], c["ks"], c["vs"], c["tables"],
                             c["lens"], scale, bound)
    assert _clean() == 0
    check(out, *_want(c, scale, out_dtype, False), "decode")


@pytest.mark.parametrize("D,B,out_dtype", [(64, 16, F32), (128, 32, BF), (128, 16, F32)])
@pytest.mark.parametrize("exponents,gap", ALL)
@pytest.mark.parametrize("more,bound", [(0, 700), (0, 5000), (0, 1100), (9000, 1100)])
def test_chunks(D, B, out_dtype, exponents, gap, more, bound):
    """Tokens by themselves, row tiles with keys in parts and with whole ones."""
    _clean()
    c = _problem([(3, 3), (5, 100), (7, 700), (2, B + 1), (4, 600)], 8, 2, D, B, BF, exponents, 32,
                 gap)
    out = torch.full(c["q"].shape, math.nan, dtype=out_dtype, device="cuda")
    scale = 1.0 / math.sqrt(D)
    pkv.paged_attn_multi_query_q8(out, c["q"].cuda(), c["q_start"], c["kp"], c["vp"], c["ks"],
                                  c["vs"], c["tables"], c["lens"], scale, 7 + more, bound)
    assert _clean() == 0
    check(out, *_want(c, scale, out_dtype, out_dtype is not F32), "chunks")


@pytest.mark.parametrize("exponents", [[None, -117], [-117], ["zero", None, None], [110, None]])
def test_long_chunks(exponents):
    """Whole key tiles that every row sees, of one kind and mixed."""
    _clean()
    c = _problem([(130, 1500), (60, 700)], 4, 2, 64, 16, FP, exponents, 33)
    for out_dtype in (BF, F32):
        out = torch.full(c["q"].shape, math.nan, dtype=out_dtype, device="cuda")
        pkv.paged_attn_multi_query_q8(out, c["q"].cuda(), c["q_start"], c["kp"], c["vp"], c["ks"],
                                      c["vs"], c["tables"], c["lens"], 0.125, 130, 1500)
        assert _clean() == 0
        check(out, *_want(c, 0.125, out_dtype, out_dtype is not F32), "chunks")


@pytest.mark.parametrize("chunk", [False, True])
def test_long_contexts_without_values(chunk):
    """Thousands of zero values under scores that rise after the first key: zeros."""
    _clean()
    H, D, B, n, m = 20, 64, 16, 16384, 1280 if chunk else 1
    blocks = n // B
    kp = torch.zeros(blocks, B, H, D, device="cuda")
    kp[..., 0] = 1.0
    # (every 43 key tiles, where a part may start, a lower key)
    kp.view(n, H, D)[::43 * 128, :, 0] = -1.0
    kp = kp.to(torch.float8_e4m3fn)
    vp = torch.zeros_like(kp)
    ks, vs = torch.ones(blocks, H, device="cuda"), torch.full((blocks, H), 2.0 ** -117, device="cuda")
    q = torch.zeros(m, H, D, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, math.nan)
    scale = 3.9 / 2 * math.log(2.0)
    if chunk:
        start = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        pkv.paged_attn_multi_query_q8(out, q, start, kp, vp, ks, vs, tables, lens, scale, m, n)
    else:
        pkv.paged_attn_decode_q8(out, q, kp, vp, ks, vs, tables, lens, scale, n)
    assert _clean() == 0
    assert (out == 0).all()


@pytest.mark.parametrize("where", [[0], [1], [0, 2], None])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 32)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_scales_of_zero(D, B, where, out_dtype):
    """Blocks of zeros whose scales are 0 (every block: None), on all routes."""
    _clean()
    seqs = [(1, 1), (1, B), (1, 3 * B + 5), (1, 600)]
    c = _problem(seqs, 8, 2, D, B, BF, [None], 34)
    for s, (_, n) in enumerate(seqs):
        for j in range(-(-n // B)) if where is None else where:
            if j * B >= n:
                continue
            b, rows = int(c["tables"][s, j]), slice(j * B, min(n, j * B + B))
            for x, pool, sc in (("k", "kp", "ks"), ("v", "vp", "vs")):
                c[pool].view(torch.uint8)[b] = 0
                c[sc][b] = 0.0
                c[x][s][rows] = 0.0
    scale = 1.0 / math.sqrt(D)
    rest = (c["kp"], c["vp"], c["ks"], c["vs"], c["tables"], c["lens"], scale)
    for bound in (600, 20000):
        out = torch.full(c["q"].shape, math.nan, dtype=out_dtype, device="cuda")
        pkv.paged_attn_decode_q8(out, c["q"].cuda(), *rest, bound)
        assert _clean() == 0
        check(out, *_want(c, scale, out_dtype, False), "decode")
    for max_q, bound in ((1, 600), (1, 5000), (9000, 1100)):
        out = torch.full(c["q"].shape, math.nan, dtype=out_dtype, device="cuda")
        pkv.paged_attn_multi_query_q8(out, c["q"].cuda(), c["q_start"], *rest, max_q, bound)
        assert _clean() == 0
        check(out, *_want(c, scale, out_dtype, out_dtype is not F32), "chunks")

"""Causal attention of chunks over 8-bit pages against the plain 64-bit form
(tests/q8_ref.py, where the tolerances are derived)."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from paged_kv_decode_26_gb300 import _lib
from tests import q8_ref as ref
from tests.cache_ref import check

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


def _problem(seqs, H, Hk, D, B, dtype, seed=1, scales="plain", gain=1.0):
    """seqs: (new tokens, context)."""
    c = ref.paged([n for _, n in seqs], B, Hk, D, seed, scales)
    g = torch.Generator().manual_seed(seed + 50)
    starts = [0]
    for m, _ in seqs:
        starts.append(starts[-1] + m)
    c["q"] = (torch.randn(starts[-1], H, D, generator=g) * gain).to(dtype)
    c["starts"] = starts
    c["q_start"] = torch.tensor(starts, dtype=torch.int32).cuda()
    return c


def _run(c, scale, out_dtype, max_q, max_len, stream=None):
    out = torch.full(c["q"].shape, 7.0, dtype=out_dtype, device="cuda")
    pkv.paged_attn_multi_query_q8(out, c["q"].cuda(), c["q_start"], c["kp"], c["vp"], c["ks"],
                                  c["vs"], c["tables"], c["lens"], scale, max_q, max_len,
                                  stream=stream)
    return out


def _want(c, scale, out_dtype, missing=None):
    """missing: per sequence, tokens that are left out."""
    q = c["q"]
    T, H, D = q.shape
    out, bound = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    for s, (a, b) in enumerate(zip(c["starts"], c["starts"][1:])):
        k, v = c["k"][s], c["v"][s]
        n, Hk = k.shape[0], k.shape[1]
        if b == a:
            continue
        G = H // Hk
        hidden = torch.ones(b - a, n, dtype=torch.bool).triu(n - (b - a) + 1)
        if missing and missing.get(s):
            hidden[:, list(missing[s])] = True
        none = hidden.all(1)
        for h in range(H):
            o, e = ref.attend_bound(q[a:b, h], k[:, h // G], v[:, h // G], scale, out_dtype, hidden,
                                    once=out_dtype is not F32, chained=True)
            o[none], e[none] = 0.0, 0.0
            out[a:b, h], bound[a:b, h] = o, e
    return out, bound


CASES = [
    # seqs (new, context), H, Hk, D, B, dtype, out
    ([(1, 1)], 1, 1, 64, 16, FP, FP),
    ([(1, 1)], 8, 1, 128, 32, BF, F32),
    ([(3, 3), (0, 0), (1, 40), (0, 5), (5, 33)], 8, 8, 64, 16, BF, BF),
    ([(127, 127), (128, 128), (129, 129)], 4, 4, 128, 16, BF, BF),
    ([(255, 300), (256, 256), (257, 400)], 2, 2, 64, 32, FP, FP),
    ([(64, 200), (33, 129), (65, 1000)], 8, 2, 128, 16, BF, BF),
    ([(100, 517), (4, 2049)], 8, 1, 128, 32, FP, F32),
    ([(31, 400), (32, 32), (33, 77), (17, 17)], 6, 3, 128, 16, BF, F32),
    ([(300, 900)], 16, 2, 64, 16, FP, FP),
    ([(40, 4000), (7, 100)], 4, 2, 128, 16, BF, BF),
    ([(2, 30)] * 70, 4, 4, 64, 16, BF, BF),
]


@pytest.mark.parametrize("seqs,H,Hk,D,B,dtype,out_dtype", CASES)
def test_multi_query_q8(seqs, H, Hk, D, B, dtype, out_dtype):
    _clean()
    c = _problem(seqs, H, Hk, D, B, dtype)
    scale = 1.0 / math.sqrt(D)
    max_q, max_len = max(m for m, _ in seqs), max(n for _, n in seqs)
    out = _run(c, scale, out_dtype, max_q, max_len)
    assert _clean() == 0
    want = _want(c, scale, out_dtype)
    check(out, *want, "chunk")
    assert torch.equal(out, _run(c, scale, out_dtype, max_q, max_len)), "not the same bits twice"
    # bounds far above the lengths: more key parts, some of them empty
    for more_q, more_len in ((0, 20000), (300, 2)):
        check(_run(c, scale, out_dtype, max_q + more_q, max_len + more_len), *want, "bounds")
    assert _clean() == 0


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 32)])
def test_scales_of_all_sizes(D, B, out_dtype):
    c = _problem([(40, 700), (9, 9)], 4, 2, D, B, BF, 3, "wide", gain=0.5)
    out = _run(c, 0.1, out_dtype, 40, 700)
    assert _clean() == 0
    check(out, *_want(c, 0.1, out_dtype), "wide scales")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gain", [2.0 ** -14, 30.0, 2000.0])
def test_queries_of_all_sizes(dtype, gain):
    c = _problem([(20, 400)], 4, 2, 64, 16, dtype, 4, gain=gain)
    out = _run(c, 0.125, F32, 20, 400)
    assert _clean() == 0
    want, bound = _want(c, 0.125, F32)
    check(out, want, bound.clamp(max=1e3), "queries")


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scale_not_positive(scale):
    c = _problem([(20, 300)], 4, 2, 64, 16, BF, 5)
    out = _run(c, scale, BF, 20, 300)
    assert _clean() == 0
    check(out, *_want(c, scale, BF), "scale")


@pytest.mark.parametrize("bound", [300, 3000])
def test_large_scores(bound):
    """Scores of 2^20 and more: formed ahead of the maximum; the largest wins."""
    c = _problem([(30, 300)], 4, 2, 128, 16, BF, 6, gain=1.0)
    out = _run(c, 2.0 ** 20, BF, 30, bound)
    assert _clean() == 0
    q, k, v = c["q"].double(), c["k"][0], c["v"][0]
    for h in range(4):
        x = q[:, h] @ k[:, h // 2].T
        x = x.masked_fill(torch.ones(30, 300, dtype=torch.bool).triu(271), -math.inf)
        best, second = x.topk(2, -1).values.unbind(-1)
        clear = best - second > 1e-3              # 2^10 in the exponent, far above fp32's error
        want = v[x.argmax(-1), h // 2]
        err = (out[:, h].double().cpu() - want).abs()
        assert clear.sum() > 20 and (err[clear] <= 2.0 ** -8 * want[clear].abs() + 1e-12).all()


def test_bf16_queries_beyond_fp16():
    c = _problem([(20, 100)], 4, 1, 64, 16, BF, 7)
    want = _run(c, 0.125, F32, 20, 100)
    q = c["q"]
    for up in (2.0 ** 60, 2.0 ** -60):
        c["q"] = (q.float() * up).to(BF)
        assert torch.equal(_run(c, 0.125 / up, F32, 20, 100), want), up
    assert _clean() == 0


@pytest.mark.parametrize("B", [16, 32])
def test_blocks_outside_the_pool_are_left_out(B):
    _clean()
    c = _problem([(50, 300), (20, 20)], 4, 2, 64, B, FP, 8)
    nb = c["kp"].shape[0]
    c["tables"][0, 1], c["tables"][0, 5], c["tables"][1, 0] = -1, nb, 1 << 30
    out = _run(c, 0.125, F32, 50, 300)
    assert _clean() == _lib.DEVERR_BLOCK_ID
    gone = {0: list(range(B, 2 * B)) + list(range(5 * B, 6 * B)), 1: range(0, min(B, 20))}
    check(out, *_want(c, 0.125, F32, gone), "missing blocks")


def test_sequences_out_of_bounds_are_left_out():
    _clean()
    seqs = [(10, 50), (20, 60), (9, 70), (5, 5)]
    c = _problem(seqs, 2, 1, 64, 16, BF, 9)
    good = _run(c, 0.1, BF, 20, 70)
    assert _clean() == 0
    c["lens"][0] = 9                                  # below its new tokens
    c["lens"][2] = 1000                               # beyond its table
    out = _run(c, 0.1, BF, 20, 70)
    assert _clean() == _lib.DEVERR_CONTEXT
    assert (out[:10] == 7.0).all() and (out[30:39] == 7.0).all()
    assert torch.equal(out[10:30], good[10:30]) and torch.equal(out[39:], good[39:])
    c["lens"][0], c["lens"][2] = 50, 70
    out = _run(c, 0.1, BF, 19, 70)                    # more new tokens than said
    assert _clean() == _lib.DEVERR_CONTEXT
    assert (out[10:30] == 7.0).all() and torch.equal(out[:10], good[:10])


@pytest.mark.parametrize("D,Hk", [(64, 2), (128, 1)])
@pytest.mark.parametrize("bound", [190, 9000])
def test_nan_reaches_the_rows_that_see_it(D, Hk, bound):
    seqs = [(60, 190), (140, 140)]
    c = _problem(seqs, 4, Hk, D, 16, BF, 10)
    clean = _run(c, 0.1, BF, 140, bound)
    hit = [(0, 3, 0, 1), (0, 150, Hk - 1, D - 1), (0, 189, 0, 40), (1, 0, 0, 9), (1, 130, 0, 33)]
    want = torch.zeros(c["q"].shape, dtype=torch.bool)
    G = 4 // Hk
    for s, t, h, d in hit:
        b = int(c["tables"][s, t // 16])
        c["vp"].view(torch.uint8)[b, t % 16, h, d] = 0xff if t % 2 else 0x7f
        first = max(0, t - (seqs[s][1] - seqs[s][0]))
        want[c["starts"][s] + first:c["starts"][s + 1], h * G:(h + 1) * G, d] = True
    out = _run(c, 0.1, BF, 140, bound)
    assert _clean() == 0
    assert torch.equal(out.isnan().cpu(), want)
    assert torch.equal(out[~want.cuda()], clean[~want.cuda()])


def test_nan_scales_of_blocks_that_a_row_does_not_see():
    """The scales of a sequence's last block are NaN: rows ahead of it do not notice."""
    c = _problem([(40, 40)], 2, 2, 64, 16, BF, 11)
    clean = _run(c, 0.1, BF, 40, 40)
    b = int(c["tables"][0, 2])
    c["ks"][b, 0] = math.nan
    c["vs"][b, 1] = math.nan
    out = _run(c, 0.1, BF, 40, 40)
    assert _clean() == 0
    assert torch.equal(out[:32], clean[:32])
    assert out[32:].isnan().all()


def test_zero_scales_of_keys():
    """A block of zero keys (the least scale) beside others, partly hidden."""
    c = _problem([(40, 40)], 2, 1, 64, 16, BF, 12)
    for j in (1, 2):
        b = int(c["tables"][0, j])
        c["kp"].view(torch.uint8)[b] = 0
        c["ks"][b] = 2.0 ** -117
        c["k"][0][16 * j:16 * j + 16] = 0
    out = _run(c, 2.0 ** -10, BF, 40, 40)
    assert _clean() == 0
    check(out, *_want(c, 2.0 ** -10, BF), "zero keys")


def test_rows_of_no_sequence_stay():
    c = _problem([(10, 50), (6, 30)], 4, 2, 64, 16, BF, 13)
    want = _run(c, 0.1, BF, 10, 50)
    c["q"] = torch.cat([c["q"][:1], c["q"], c["q"][:3]])
    c["q_start"] += 1
    out = _run(c, 0.1, BF, 10, 50)
    assert _clean() == 0
    assert torch.equal(out[1:17], want) and (out[:1] == 7.0).all() and (out[17:] == 7.0).all()


def test_longest_first_order_and_pools_beyond_4_gb():
    """Contexts long enough that CTAs rank the sequences, in a pool whose byte
    offsets pass 32 bits; some rows against the 64-bit form."""
    _clean()
    Hk, D, B = 8, 128, 16
    blocks = 280000                                  # 4.6 GB each
    g = torch.Generator(device="cuda").manual_seed(14)
    kp, vp = (torch.randint(64, 120, (blocks, B, Hk, D), generator=g, device="cuda",
                            dtype=torch.uint8) for _ in range(2))
    sign = torch.randint(0, 2, (1, B, Hk, D), generator=g, device="cuda", dtype=torch.uint8) << 7
    kp, vp = (kp | sign).view(torch.float8_e4m3fn), (vp | sign).view(torch.float8_e4m3fn)
    ks, vs = (torch.rand(blocks, Hk, generator=g, device="cuda") / 1000 + 1e-3 for _ in range(2))
    seqs = [(40, 700), (3, 9000), (64, 5000)]
    lens = torch.tensor([n for _, n in seqs], dtype=torch.int32).cuda()
    width = max(-(-n // B) for _, n in seqs)
    tables = torch.randperm(blocks, generator=g, device="cuda").flip(0)[:3 * width].to(torch.int32)
    tables = (blocks - 1 - tables % 4000).view(3, width).contiguous()      # the pool's end
    starts = [0, 40, 43, 107]
    q = torch.randn(107, Hk, D, generator=g, device="cuda").to(BF)
    out = torch.full((107, Hk, D), 7.0, dtype=BF, device="cuda")
    pkv.paged_attn_multi_query_q8(out, q, torch.tensor(starts, dtype=torch.int32).cuda(), kp, vp, ks,
                                  vs, tables, lens, 0.02, 64, 9000)
    assert _clean() == 0
    for s, (m, n) in enumerate(seqs):
        b = tables[s].long()
        k, v = ((p.view(torch.uint8)[b].view(torch.float8_e4m3fn).float().double()
                 * sc[b].double()[:, None, :, None]).flatten(0, 1)[:n].cpu()
                for p, sc in ((kp, ks), (vp, vs)))
        hidden = torch.ones(m, n, dtype=torch.bool).triu(n - m + 1)
        for h in (0, 5):
            o, e = ref.attend_bound(q[starts[s]:starts[s + 1], h].cpu(), k[:, h], v[:, h], 0.02, BF,
                                    hidden, once=True, chained=True)
            check(out[starts[s]:starts[s + 1], h], o, e, f"sequence {s} head {h}")


@pytest.mark.parametrize("bound,parts", [(600, False), (3000, True)])
def test_streams_graphs_and_workspaces(bound, parts):
    c = _problem([(30, 200), (5, 600)], 8, 2, 128, 16, BF, 15)
    want = _run(c, 0.1, BF, 30, bound)
    n = pkv.multi_query_q8_workspace_bytes(2, 30, 8, 2, 128, 16, bound)
    assert (n > 0) == parts          # keys in parts meet in the workspace
    q = c["q"].cuda()
    outs, graphs = [], []
    for i in range(2):
        out = torch.zeros_like(want)
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_attn_multi_query_q8(out, q, c["q_start"], c["kp"], c["vp"], c["ks"], c["vs"],
                                          c["tables"], c["lens"], 0.1, 30, bound, workspace=ws)
        outs.append((out, ws))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for s in streams:
        s.synchronize()
    third = _run(c, 0.1, BF, 30, bound, streams[0])
    streams[0].synchronize()
    assert _clean() == 0
    for out in (outs[0][0], outs[1][0], third):
        assert torch.equal(out, want)
    if not parts:
        return
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attn_multi_query_q8(out, q, c["q_start"], c["kp"], c["vp"], c["ks"], c["vs"],
                                      c["tables"], c["lens"], 0.1, 30, bound, workspace=ws[:256])


# more pairs of row tiles than a GPU has SMs; the first three: the rest of them in parts
MANY = [
    ([(300, n) for n in (1400, 300, 2500, 513, 2000)], 32, 32, 64, 16, BF, BF),
    ([(130, n) for n in (3000, 130, 1111, 2900)], 64, 16, 128, 32, FP, F32),
    ([(40, 2000 + 7 * i) for i in range(10)], 64, 16, 64, 16, BF, F32),
    ([(300, 1400), (1, 1), (0, 5), (257, 2500), (130, 600)], 32, 32, 64, 16, BF, BF),
    ([(3, 700 + 3 * i) for i in range(60)], 8, 4, 64, 16, FP, FP),
    ([(1 + i % 3, 3 + i % 50) for i in range(600)], 2, 2, 64, 32, BF, BF),
]


@pytest.mark.parametrize("seqs,H,Hk,D,B,dtype,out_dtype", MANY)
def test_many_row_tiles(seqs, H, Hk, D, B, dtype, out_dtype):
    c = _problem(seqs, H, Hk, D, B, dtype, 20)
    scale = 1.0 / math.sqrt(D)
    max_q, max_len = max(m for m, _ in seqs), max(n for _, n in seqs)
    out = _run(c, scale, out_dtype, max_q, max_len)
    assert _clean() == 0
    want = _want(c, scale, out_dtype)
    check(out, *want, "many row tiles")
    assert torch.equal(out, _run(c, scale, out_dtype, max_q, max_len)), "not the same bits twice"
    check(_run(c, scale, out_dtype, max_q + 300, max_len + 9000), *want, "bounds")
    check(_run(c, scale, out_dtype, max_q, 9000), *want, "longest first")
    assert _clean() == 0


EQUAL = [(257, n) for n in (1400, 600, 2500, 1000, 2400)]


@pytest.mark.parametrize("gone", [1, 4])
def test_what_is_left_of_many_row_tiles(gone):
    """A sequence that does not fit its bounds, missing blocks and NaN beside parts."""
    H, B = 32, 16
    c = _problem(EQUAL, H, H, 64, B, BF, 21)
    nb, starts = c["kp"].shape[0], c["starts"]
    assert pkv.multi_query_q8_workspace_bytes(5, 257, H, H, 64, B, 2500) > 0
    _clean()
    c["lens"][gone] = 256
    c["tables"][0, 40], c["tables"][2, 3] = -1, nb
    missing = {0: range(40 * B, 41 * B), 2: range(3 * B, 4 * B)}
    if gone != 4:
        c["tables"][4, 100] = -1
        missing[4] = range(100 * B, 101 * B)
    out = _run(c, 0.125, BF, 257, 2500)
    assert _clean() == _lib.DEVERR_CONTEXT | _lib.DEVERR_BLOCK_ID
    own = slice(starts[gone], starts[gone + 1])
    assert (out[own] == 7.0).all()
    want, bound = _want(c, 0.125, BF, missing)
    want[own], bound[own] = 7.0, 0.0
    check(out, want, bound, "what is left")
    nan = torch.zeros(out.shape, dtype=torch.bool)
    for s, t, h, d in ((0, 1399, 5, 3), (0, 20, 31, 63), (2, 2499, 0, 0), (4, 2200, 17, 9),
                       (4, 9, 31, 1)):
        if s == gone:
            continue
        b = int(c["tables"][s, t // B])
        c["vp"].view(torch.uint8)[b, t % B, h, d] = 0x7f
        first = max(0, t - (EQUAL[s][1] - EQUAL[s][0]))
        nan[starts[s] + first:starts[s + 1], h, d] = True
    hit = _run(c, 0.125, BF, 257, 2500)
    _clean()
    assert torch.equal(hit.isnan().cpu(), nan)
    assert torch.equal(hit[~nan.cuda()], out[~nan.cuda()])


def test_streams_graphs_of_many_row_tiles():
    c = _problem(EQUAL, 32, 32, 64, 16, BF, 22)
    want = _run(c, 0.1, BF, 257, 2500)
    n = pkv.multi_query_q8_workspace_bytes(5, 257, 32, 32, 64, 16, 2500)
    assert n > 0
    q = c["q"].cuda()
    outs, graphs = [], []
    for i in range(2):
        out, ws = torch.zeros_like(want), torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_attn_multi_query_q8(out, q, c["q_start"], c["kp"], c["vp"], c["ks"], c["vs"],
                                          c["tables"], c["lens"], 0.1, 257, 2500, workspace=ws)
        outs.append((out, ws))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert _clean() == 0
    for out, _ in outs:
        assert torch.equal(out, want)
    # other lengths at the next replay
    c["lens"].copy_(torch.tensor([700, 257, 300, 599, 1500], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], _run(c, 0.1, BF, 257, 2500))


FEW = [(1, 1), (7, 7), (8, 8), (9, 33), (2, 32), (3, 31), (8, 64), (5, 65), (0, 9), (6, 1000), (4, 35)]


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 32)])
def test_few_tokens(D, B, G, out_dtype):
    """Tokens of a sequence as columns of one product (the second bound: row tiles)."""
    c = _problem(FEW, G, 1, D, B, BF, 23)
    for bound in (5000, 1000):
        out = _run(c, 0.1, out_dtype, 9, bound)
        assert _clean() == 0
        check(out, *_want(c, 0.1, out_dtype), f"few tokens, bound {bound}")
    # NaN in values of the last tokens, and in the scale of a block that only they reach
    nan = torch.zeros(c["q"].shape, dtype=torch.bool)
    for s, t, d in ((0, 0, 3), (2, 7, 0), (3, 32, D - 1), (3, 30, 1), (7, 63, 5), (7, 64, 5),
                    (9, 995, 2), (9, 10, 9), (10, 31, 40), (10, 32, 41), (10, 34, 42)):
        b = int(c["tables"][s, t // B])
        c["vp"].view(torch.uint8)[b, t % B, 0, d] = 0xff
        m, n = FEW[s]
        nan[c["starts"][s] + max(0, t - (n - m)):c["starts"][s + 1], :, d] = True
    hit = _run(c, 0.1, out_dtype, 9, 1000)
    assert torch.equal(hit.isnan().cpu(), nan)
    assert torch.equal(hit[~nan.cuda()], out[~nan.cuda()])
    last = int(c["tables"][3, 32 // B])              # holds token 32 alone
    c["vs"][last, 0] = math.nan
    again = _run(c, 0.1, out_dtype, 9, 1000)
    assert _clean() == 0
    own = slice(c["starts"][3] + 8, c["starts"][4])  # the one token that sees it
    nan[own] = True
    assert torch.equal(again.isnan().cpu(), nan)
    assert torch.equal(again[~nan.cuda()], hit[~nan.cuda()])


def test_few_tokens_of_missing_blocks():
    c = _problem([(6, 40), (3, 20), (5, 70)], 4, 2, 64, 16, FP, 24)
    nb = c["kp"].shape[0]
    _clean()
    c["tables"][0, 2], c["tables"][2, 1] = nb, -1    # the last block of the first
    c["lens"][1] = 2                                 # below its new tokens
    out = _run(c, 0.1, F32, 6, 70)
    assert _clean() == _lib.DEVERR_BLOCK_ID | _lib.DEVERR_CONTEXT
    want, bound = _want(c, 0.1, F32, {0: range(32, 40), 2: range(16, 32)})
    want[6:9], bound[6:9] = 7.0, 0.0
    check(out, want, bound, "missing blocks")


def test_one_token_is_the_decode():
    lens = [300, 17, 1]
    c = _problem([(1, n) for n in lens], 8, 2, 64, 16, FP, 16)
    out = _run(c, 0.125, F32, 1, 300)
    dec = torch.empty_like(out)
    pkv.paged_attn_decode_q8(dec, c["q"].cuda(), c["kp"], c["vp"], c["ks"], c["vs"], c["tables"],
                             c["lens"], 0.125, 300)
    assert _clean() == 0
    want, bound = _want(c, 0.125, F32)
    assert ((out - dec).double().cpu().abs() <= 2 * bound).all()


def test_binding_refusals():
    c = _problem([(3, 20)], 4, 2, 64, 16, BF, 17)
    q = c["q"].cuda()
    out = torch.empty_like(q)
    ok = [out, q, c["q_start"], c["kp"], c["vp"], c["ks"], c["vs"], c["tables"], c["lens"], 0.1, 3, 20]
    for i, bad in ((0, out[:, :2]), (1, q.cpu()), (2, c["q_start"].long()), (2, c["q_start"][:1]),
                   (3, c["kp"].view(torch.uint8)), (4, c["vp"][:1].clone()), (5, c["ks"].double()),
                   (6, c["vs"][:1]), (7, c["tables"].long()), (8, c["lens"].cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            pkv.paged_attn_multi_query_q8(*args)
    assert _clean() == 0

"""Decode over 8-bit pages against the plain 64-bit form (tests/q8_ref.py, where
the tolerances are derived)."""
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


def _q(S, H, D, dtype, seed=2, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(S, H, D, generator=g) * gain).to(dtype)


def _want(c, q, scale, out_dtype):
    S, H, D = q.shape
    out, bound = torch.zeros(S, H, D, dtype=torch.float64), torch.zeros(S, H, D, dtype=torch.float64)
    for s in range(S):
        Hk = c["k"][s].shape[1]
        G = H // Hk
        for j in range(Hk):
            h = slice(j * G, (j + 1) * G)
            out[s, h], bound[s, h] = ref.attend_bound(q[s, h], c["k"][s][:, j], c["v"][s][:, j],
                                                      scale, out_dtype)
    return out, bound


def _run(c, q, scale, out_dtype, max_len, **kw):
    out = torch.full(q.shape, math.nan, dtype=out_dtype, device="cuda")
    pkv.paged_attn_decode_q8(out, q.cuda(), c["kp"], c["vp"], c["ks"], c["vs"], c["tables"],
                             c["lens"], scale, max_len, **kw)
    return out


CASES = [
    # lens, H, Hk, D, B, dtype, out
    ([1], 1, 1, 64, 16, FP, F32),
    ([0, 1, 15, 16, 17, 0, 31, 32, 33], 8, 8, 128, 16, BF, BF),
    ([200, 3, 77, 0], 8, 8, 64, 16, FP, F32),
    ([31, 32, 33, 500], 8, 2, 128, 32, BF, F32),
    ([1000, 1, 64], 6, 3, 128, 16, BF, BF),
    ([700, 2], 24, 12, 64, 32, FP, FP),
    ([129] * 40 + [0, 5], 16, 2, 64, 16, BF, BF),
    ([5000, 11, 2500], 32, 8, 128, 16, BF, BF),
    ([9000], 8, 1, 128, 32, FP, F32),
    ([7, 300, 0, 0, 45, 1, 1, 1, 90] * 60, 4, 4, 64, 16, BF, F32),
    ([300] * 300, 32, 32, 64, 16, FP, FP),
]


@pytest.mark.parametrize("lens,H,Hk,D,B,dtype,out_dtype", CASES)
def test_decode_q8(lens, H, Hk, D, B, dtype, out_dtype):
    _clean()
    c = ref.paged(lens, B, Hk, D, 1)
    q = _q(len(lens), H, D, dtype)
    scale = 1.0 / math.sqrt(D)
    want = _want(c, q, scale, out_dtype)
    # (a bound far above the lengths: in pieces, even where contexts are short)
    for max_len in (max(lens) + 3, 20000):
        out = _run(c, q, scale, out_dtype, max_len)
        assert _clean() == 0
        check(out, *want, f"decode, bound {max_len}")
        again = _run(c, q, scale, out_dtype, max_len)
        assert torch.equal(out, again), "not the same bits twice"


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 32)])
def test_scales_of_all_sizes(D, B, out_dtype):
    """Value scales 2^-16 .. 2^8 from block to block: the weights' reference moves."""
    lens = [700, 40, 16, 1]
    c = ref.paged(lens, B, 2, D, 3, scales="wide")
    q = _q(4, 4, D, BF, gain=0.5)
    for max_len in (700, 7000):
        out = _run(c, q, 0.1, out_dtype, max_len)
        assert _clean() == 0
        check(out, *_want(c, q, 0.1, out_dtype), f"wide scales, bound {max_len}")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gain", [2.0 ** -14, 30.0, 2000.0])
def test_queries_of_all_sizes(dtype, gain):
    lens = [400, 33]
    c = ref.paged(lens, 16, 2, 64, 4)
    q = _q(2, 16, 64, dtype, gain=gain)
    out = _run(c, q, 0.125, F32, 400)
    assert _clean() == 0
    want, bound = _want(c, q, 0.125, F32)
    # (where scores are that large a weight's bound may be beyond 1)
    check(out, want, bound.clamp(max=1e3), "queries")


def test_bf16_queries_beyond_fp16():
    lens = [100]
    c = ref.paged(lens, 16, 1, 64, 5)
    q = _q(1, 4, 64, BF, gain=1.0)
    want = _run(c, q, 2.0 ** -3, F32, 100)
    for up in (2.0 ** 60, 2.0 ** -60):
        got = _run(c, (q.float() * up).to(BF), 2.0 ** -3 / up, F32, 100)
        assert torch.equal(got, want), up
    assert _clean() == 0


def test_blocks_outside_the_pool_are_left_out():
    _clean()
    lens = [100, 64, 20]
    for B in (16, 32):
        c = ref.paged(lens, B, 2, 64, 6)
        n_blocks = c["kp"].shape[0]
        q = _q(3, 4, 64, FP)
        c["tables"][0, 1], c["tables"][1, 0], c["tables"][2, 0] = -1, n_blocks, 1 << 30
        out = _run(c, q, 0.125, F32, 100)
        assert _clean() == _lib.DEVERR_BLOCK_ID
        pieces = _run(c, q, 0.125, F32, 3000)
        assert _clean() == _lib.DEVERR_BLOCK_ID
        gone = {0: range(B, 2 * B), 1: range(0, B), 2: range(0, min(B, 20))}
        for s, rows in gone.items():
            keep = [t for t in range(lens[s]) if t not in rows]
            c["k"][s], c["v"][s] = c["k"][s][keep], c["v"][s][keep]
        check(out, *_want(c, q, 0.125, F32), "missing blocks")
        check(pieces, *_want(c, q, 0.125, F32), "missing blocks, in pieces")


def test_lengths_out_of_bounds():
    _clean()
    c = ref.paged([50, 60, 70], 16, 1, 64, 7)
    q = _q(3, 2, 64, BF)
    c["lens"][1], c["lens"][2] = -3, 1000
    out = _run(c, q, 0.1, F32, 64)
    assert _clean() == _lib.DEVERR_CONTEXT
    c["k"][1], c["v"][1] = c["k"][1][:0], c["v"][1][:0]
    c["k"][2], c["v"][2] = c["k"][2][:64], c["v"][2][:64]
    check(out, *_want(c, q, 0.1, F32), "clamped")


def test_nan_in_the_cache_reaches_its_own_sequence_and_head():
    c = ref.paged([40, 40], 16, 2, 64, 8)
    q = _q(2, 4, 64, BF)
    b = int(c["tables"][0, 1])
    c["vp"].view(torch.uint8)[b, 3, 1, 5] = 0x7f
    want = torch.zeros(2, 4, 64, dtype=torch.bool)
    want[0, 2:, 5] = True
    for max_len in (40, 4000):
        out = _run(c, q, 0.1, F32, max_len)
        assert _clean() == 0
        assert torch.equal(out.isnan().cpu(), want)


def test_empty_pool_and_empty_contexts():
    q = _q(3, 4, 64, BF).cuda()
    out = torch.full((3, 4, 64), math.nan, dtype=BF, device="cuda")
    e = torch.zeros(0, 16, 2, 64, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.zeros(0, 2, device="cuda")
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    pkv.paged_attn_decode_q8(out, q, e, e, sc, sc, torch.zeros(3, 1, dtype=torch.int32, device="cuda"),
                             z, 0.1, 0)
    assert _clean() == 0 and (out == 0).all()
    pkv.paged_attn_decode_q8(out[:0], q[:0], e, e, sc, sc,
                             torch.zeros(0, 1, dtype=torch.int32, device="cuda"), z[:0], 0.1, 0)


def test_taken_over_runs_and_pools_beyond_4_gb():
    """A batch large enough that CTAs take over short runs, in a pool whose byte
    offsets pass 32 bits; a few sequences against the 64-bit form."""
    _clean()
    S, Hk, D, B, n = 64, 32, 128, 32, 3200
    pages = n // B
    blocks = 36000                                  # 4.7 GB each
    g = torch.Generator(device="cuda").manual_seed(9)
    kp, vp = (torch.randint(0, 120, (blocks, B, Hk, D), generator=g, device="cuda",
                            dtype=torch.uint8) for _ in range(2))
    kp |= torch.randint(0, 2, (1, B, Hk, D), generator=g, device="cuda", dtype=torch.uint8) << 7
    kp, vp = kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
    ks, vs = (torch.rand(blocks, Hk, generator=g, device="cuda") / 100 + 1e-3 for _ in range(2))
    tables = torch.randperm(blocks, generator=g, device="cuda")[-S * pages:].to(torch.int32)
    tables = tables.view(S, pages).contiguous()
    lens = torch.randint(n - 500, n + 1, (S,), generator=g, device="cuda").to(torch.int32)
    q = _q(S, Hk, D, BF)
    out = torch.full((S, Hk, D), math.nan, dtype=F32, device="cuda")
    pkv.paged_attn_decode_q8(out, q.cuda(), kp, vp, ks, vs, tables, lens, 0.05, n)
    assert _clean() == 0
    for s in (0, 31, 63):
        m = int(lens[s])
        b = tables[s].long()
        k, v = ((p.view(torch.uint8)[b].view(torch.float8_e4m3fn).float().double()
                 * sc[b].double()[:, None, :, None]).flatten(0, 1)[:m].cpu()
                for p, sc in ((kp, ks), (vp, vs)))
        for h in (0, 13, 31):
            o, bound = ref.attend_bound(q[s, h:h + 1], k[:, h], v[:, h], 0.05, F32)
            check(out[s, h:h + 1], o, bound, f"sequence {s} head {h}")


@pytest.mark.parametrize("bound", [512, 5000])
def test_streams_graphs_and_workspaces(bound):
    lens = [500, 20, 0, 333]
    c = ref.paged(lens, 16, 2, 128, 10)
    q = _q(4, 8, 128, BF).cuda()
    want = _run(c, q.cpu(), 0.1, BF, bound)
    n = pkv.decode_q8_workspace_bytes(4, 8, 2, 128, 16, bound)
    outs, graphs = [], []
    for i in range(2):
        out = torch.zeros_like(want)
        ws = torch.full((max(n, 256),), 0xff, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attn_decode_q8(out, q, c["kp"], c["vp"], c["ks"], c["vs"], c["tables"],
                                     c["lens"], 0.1, bound, workspace=ws)
        outs.append((out, ws))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for s in streams:
        s.synchronize()
    third = _run(c, q.cpu(), 0.1, BF, bound, stream=streams[0])
    streams[0].synchronize()
    assert _clean() == 0
    for out in (outs[0][0], outs[1][0], third):
        assert torch.equal(out, want)


def test_appended_cache_decodes_as_its_values():
    """Tokens appended step by step, then decoded: the 8-bit decode against the
    16-bit decode of the values that the pages stand for."""
    S, H, Hk, D, B, steps = 3, 8, 2, 64, 16, 40
    g = torch.Generator().manual_seed(11)
    blocks = S * 4
    bm = pkv.BlockManager(blocks, B)
    tables = torch.full((S, 4), -1, dtype=torch.int32)
    lens = torch.zeros(S, dtype=torch.int32)
    slots = torch.empty(S, dtype=torch.int64)
    kp, vp = (torch.zeros(blocks, B, Hk, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(blocks, Hk, device="cuda") for _ in range(2))
    rope = pkv.rope_table(torch.empty(64, D, device="cuda"), pkv.rope_frequencies(D)[0])
    q_out = torch.empty(S, H, D, dtype=FP, device="cuda")
    out, out16 = torch.empty(S, H, D, device="cuda"), torch.empty(S, H, D, device="cuda")
    for step in range(steps):
        assert bm.append_slots(tables, lens, slots) == 0
        qkv = torch.randn(S, H + 2 * Hk, D, generator=g).to(FP).cuda()
        pkv.kv_append_rope_q8(kp, vp, ks, vs, qkv[:, H:H + Hk], qkv[:, H + Hk:], slots.cuda(),
                              (lens - 1).cuda(), rope, qkv[:, :H], q_out)
        pkv.paged_attn_decode_q8(out, q_out, kp, vp, ks, vs, tables.cuda(), lens.cuda(), 0.125, steps)
        # (powers of two: the values are fp16 numbers)
        k16, v16 = ((p.float() * sc[:, None, :, None]).to(FP) for p, sc in ((kp, ks), (vp, vs)))
        pkv.paged_attn_decode(out16, q_out, k16, v16, tables.cuda(), lens.cuda(), 0.125, steps)
        assert (out - out16).abs().max() <= 2e-5, step
    assert _clean() == 0


def test_binding_refusals():
    c = ref.paged([20], 16, 2, 64, 12)
    q = _q(1, 4, 64, BF).cuda()
    out = torch.empty_like(q)
    ok = [out, q, c["kp"], c["vp"], c["ks"], c["vs"], c["tables"], c["lens"], 0.1, 20]
    for i, bad in ((0, out[:, :2]), (1, q.cpu()), (2, c["kp"].view(torch.uint8)),
                   (3, c["vp"][:1].clone()), (4, c["ks"].double()), (5, c["vs"][:1]),
                   (5, c["vs"][:, :1].contiguous()), (6, c["tables"].long()), (7, c["lens"].cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            pkv.paged_attn_decode_q8(*args)
    ok[-1] = 5000
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attn_decode_q8(*ok, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert _clean() == 0

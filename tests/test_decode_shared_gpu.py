"""paged_attn_decode_shared against a plain 64-bit form of the ordinary decode
(tests/cache_ref.py, where the tolerances are derived; the prefix's softmax
weights are rounded once for 16-bit outputs)."""
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


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _problem(lens, starts, prefix, H, Hk, D, B, dtype, seed=1):
    c = ref.paged(lens, B, Hk, D, dtype, seed, shared=(starts, prefix))
    g = torch.Generator().manual_seed(seed + 100)
    c["q"] = torch.randn(len(lens), H, D, generator=g).to(dtype)
    c["scale"] = 1.0 / math.sqrt(D)
    return c


def _run(c, starts, prefix, out_dtype, L, max_group=None, max_prefix=None, **kw):
    out = torch.full(c["q"].shape, float("nan"), dtype=out_dtype, device="cuda")
    sizes = [b - a for a, b in zip(starts, starts[1:])]
    pkv.paged_attn_decode_shared(
        out, c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"], c["lens"], _ints(starts),
        _ints(prefix), c["scale"], L, max(sizes + [0]) if max_group is None else max_group,
        max(prefix + [0]) if max_prefix is None else max_prefix, **kw)
    return out


CASES = [
    # lens, group starts, prefixes, H, Hk, D, B, dtype, out
    ([17], [0, 1], [16], 1, 1, 64, 16, FP, F32),
    ([16, 16], [0, 2], [16], 8, 8, 128, 16, BF, BF),                 # nothing behind the prefix
    ([65, 80, 64, 200], [0, 4], [64], 8, 8, 64, 16, FP, F32),
    ([40, 0, 33, 5, 32], [0, 5], [32], 4, 2, 128, 32, BF, BF),       # members shorter than it
    ([300, 290, 1000, 64, 70, 80], [0, 3, 6], [256, 48], 8, 2, 128, 16, BF, BF),
    ([100, 90, 80, 70], [1, 3], [64], 8, 1, 64, 16, BF, F32),        # first and last in no group
    ([50, 60], [0, 2], [0], 4, 4, 128, 16, BF, BF),                  # empty prefix
    ([50, 60, 70], [0, 0, 3, 3], [16, 48, 32], 6, 3, 64, 16, FP, FP),  # empty groups
    ([2100 + i for i in range(70)], [0, 70], [2048], 32, 8, 128, 16, BF, BF),   # 280 rows
    ([530 + 3 * i for i in range(40)], [0, 40], [512], 8, 8, 64, 32, FP, F32),
    ([129 + i for i in range(300)], list(range(0, 301, 3)), [128] * 100, 4, 4, 64, 16, BF, BF),
    ([1500, 1400, 1400], [0, 3], [1392], 16, 2, 128, 16, BF, F32),   # a short last key tile
    ([20] * 1100, list(range(1101)), [16] * 1100, 1, 1, 64, 16, BF, F32),   # many groups
]


@pytest.mark.parametrize("lens,starts,prefix,H,Hk,D,B,dtype,out_dtype", CASES)
def test_decode_shared(lens, starts, prefix, H, Hk, D, B, dtype, out_dtype):
    _clean()
    c = _problem(lens, starts, prefix, H, Hk, D, B, dtype)
    out = _run(c, starts, prefix, out_dtype, max(lens))
    assert _clean() == 0
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], out_dtype, once=out_dtype != F32)
    ref.check(out, o, bound)


def test_decode_shared_without_groups():
    _clean()
    lens = [70, 0, 300, 5]
    c = _problem(lens, [0], [], 8, 2, 128, 16, BF)
    out = _run(c, [0], [], BF, 300)
    assert _clean() == 0
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], BF)
    ref.check(out, o, bound)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_decode_shared_scales(scale):
    starts, prefix, lens = [0, 3], [160], [170, 200, 165]
    c = _problem(lens, starts, prefix, 8, 2, 64, 16, BF)
    c["scale"] = scale
    out = _run(c, starts, prefix, F32, 200)
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], scale, F32)
    ref.check(out, o, bound, f"scale {scale}")


def test_decode_shared_flags_and_decodes_alone():
    """Groups that are not well formed: flagged, and the members' results are
    those of whole contexts."""
    lens = [70, 80, 90, 100]
    for starts, prefix, mg, mp in (([0, 4], [50], 4, 64),        # no whole blocks
                                   ([0, 4], [64], 3, 64),        # more members than max_group
                                   ([0, 4], [80], 4, 64),        # beyond max_prefix
                                   ([0, 5], [64], 4, 64),        # beyond the batch
                                   ([0, 4], [-16], 4, 64)):
        _clean()
        c = _problem(lens, [0, 4], [64], 4, 2, 64, 16, BF)
        out = _run(c, starts, prefix, BF, 100, max_group=mg, max_prefix=mp)
        assert _clean() == _lib.DEVERR_CONTEXT
        o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], BF)
        ref.check(out, o, bound, str((starts, prefix)))


def test_decode_shared_flags_a_missing_page():
    _clean()
    lens, starts, prefix = [700, 600, 40], [0, 2], [512]
    c = _problem(lens, starts, prefix, 4, 2, 64, 16, BF)
    c["tables"][0, 3] = -1
    out = _run(c, starts, prefix, BF, 700)
    assert _clean() == _lib.DEVERR_BLOCK_ID
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], BF)
    ref.check(out[2:], o[2:], bound[2:])
    assert torch.isfinite(out).all()


def test_decode_shared_repeats_graph_stream():
    lens, starts, prefix = [700, 600, 40, 530], [0, 2, 4], [512, 32]
    c = _problem(lens, starts, prefix, 8, 2, 128, 16, BF)
    n = pkv.decode_shared_workspace_bytes(4, 2, 2, 512, 8, 2, 128, 16, 700)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want = _run(c, starts, prefix, BF, 700, workspace=ws)
    torch.cuda.synchronize()
    ws.fill_(255)
    assert torch.equal(_run(c, starts, prefix, BF, 700, workspace=ws), want)
    q, gs, pl = c["q"].cuda(), _ints(starts), _ints(prefix)
    out = torch.empty_like(want)
    call = lambda **kw: pkv.paged_attn_decode_shared(  # noqa: E731
        out, q, c["k_pool"], c["v_pool"], c["tables"], c["lens"], gs, pl, c["scale"], 700, 2, 512,
        workspace=ws, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("max_group,max_prefix", [(4, 0), (0, 64), (0, 0)])
def test_decode_shared_flags_groups_where_no_bound_allows_any(max_group, max_prefix):
    _clean()
    lens, starts, prefix = [70, 80, 90, 100], [0, 4], [64]
    c = _problem(lens, starts, prefix, 4, 2, 64, 16, BF)
    out = _run(c, starts, prefix, BF, 100, max_group=max_group, max_prefix=max_prefix)
    assert _clean() == _lib.DEVERR_CONTEXT
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], BF)
    ref.check(out, o, bound)


def test_decode_shared_flags_one_group_of_many():
    """More groups than a CTA keeps in shared memory, one of them malformed."""
    S = 1300
    lens = [20 + i % 30 for i in range(S)]
    starts, prefix = list(range(S + 1)), [16] * S
    c = _problem(lens, starts, prefix, 1, 1, 64, 16, BF)
    prefix[1234] = 17
    out = _run(c, starts, prefix, BF, 50, max_prefix=32)
    assert _clean() == _lib.DEVERR_CONTEXT
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], BF, once=True)
    ref.check(out, o, bound)


def test_decode_shared_from_an_empty_pool():
    """No blocks at all: the tables' ids are flagged, the rows are zeros."""
    _clean()
    q = torch.randn(2, 4, 64, device="cuda").to(BF)
    out = torch.full((2, 4, 64), 7.0, dtype=BF, device="cuda")
    pool = torch.empty(0, 16, 2, 64, dtype=BF, device="cuda")
    tables = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    pkv.paged_attn_decode_shared(out, q, pool, pool, tables, _ints([40, 50]), _ints([0, 2]),
                                 _ints([32]), 0.1, 64, 2, 32)
    assert _clean() == _lib.DEVERR_BLOCK_ID
    assert (out == 0).all()

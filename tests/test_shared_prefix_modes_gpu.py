"""paged_attn_decode_shared with its prefixes attended once per group and, by the
tuning knob, by every member alone: both against the 64-bit form at every case,
whatever the automatic choice would be (tolerances: tests/cache_ref.py)."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from paged_kv_decode_26_gb300 import _lib
from tests import cache_ref as ref
from tests import test_decode_shared_gpu as base
from tests.test_long_sums_gpu import _ints, _same_pages
from tests.test_small_weights_gpu import KINDS, _check, _paged

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(params=[0, 1], ids=["alone", "once"])
def mode(request):
    pkv.set_tuning(shared_prefix=request.param)
    yield request.param
    pkv.reset_tuning()


@pytest.mark.parametrize("lens,starts,prefix,H,Hk,D,B,dtype,out_dtype", base.CASES)
def test_both_ways(mode, lens, starts, prefix, H, Hk, D, B, dtype, out_dtype):
    base.test_decode_shared(lens, starts, prefix, H, Hk, D, B, dtype, out_dtype)


def test_both_ways_flag_bad_groups_and_pages(mode):
    base.test_decode_shared_flags_and_decodes_alone()
    base.test_decode_shared_flags_a_missing_page()
    base.test_decode_shared_flags_one_group_of_many()
    base.test_decode_shared_from_an_empty_pool()
    base.test_decode_shared_without_groups()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_both_ways_at_scales(mode, scale):
    base.test_decode_shared_scales(scale)


def test_both_ways_repeat_in_graphs_and_on_streams(mode):
    base.test_decode_shared_repeats_graph_stream()


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_once_keeps_small_weights(mode, D, dtype, out_dtype):
    n, H, Hk = 3000, 4, 2
    q, k, v, kp, vp, tables, lens = _paged(n, H, Hk, D, dtype, 3, 2000)
    out = torch.empty(3, H, D, dtype=out_dtype, device="cuda")
    pkv.paged_attn_decode_shared(out, q.cuda(), kp, vp, tables, lens, _ints([0, 3]), _ints([2000]),
                                 1.0, n, 3, 2000)
    o, bound, _ = ref.decode(q, [k] * 3, [v] * 3, 1.0, out_dtype, once=out_dtype != F32)
    _check(out, o, bound, dtype, n, "out")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_once_over_long_prefixes(mode, D, dtype):
    n, S, scale = 16000, 304, 0.5 / math.sqrt(D)
    q, k, v, qd, kp, vp, tables, lens = _same_pages(S, n, D, dtype)
    out = torch.empty(S, 2, D, dtype=F32, device="cuda")
    pkv.paged_attn_decode_shared(out, qd, kp, vp, tables, lens, _ints(list(range(S + 1))),
                                 _ints([n - 32] * S), scale, n, 1, n - 32)
    o, bound, _ = ref.decode(q, [k], [v], scale, F32)
    ref.check(out, o.expand(S, 2, D), bound, "out")


def test_workspace_covers_either_way():
    """The bytes follow the choice: a buffer for one is checked by the other."""
    need = {}
    for k in (0, 1):
        pkv.set_tuning(shared_prefix=k)
        need[k] = pkv.decode_shared_workspace_bytes(8, 1, 8, 1024, 8, 8, 64, 16, 1100)
    pkv.reset_tuning()
    assert need[0] < need[1]
    assert pkv.decode_shared_workspace_bytes(8, 1, 8, 1024, 8, 8, 64, 16, 1100) in need.values()
    c = base._problem([1060] * 8, [0, 8], [1024], 8, 8, 64, 16, BF)
    ws = torch.empty(need[0], dtype=torch.uint8, device="cuda")
    pkv.set_tuning(shared_prefix=1)
    try:
        with pytest.raises(pkv.PagedKVError) as e:
            base._run(c, [0, 8], [1024], BF, 1100, workspace=ws)
        assert e.value.status == _lib.PKV_ERR_WORKSPACE
    finally:
        pkv.reset_tuning()


@pytest.mark.parametrize("groups,H", [(60, 32), (400, 8)])
def test_items_beyond_the_sms_in_a_graph(groups, H):
    """More prefix items than SMs, taken over by running CTAs (480), and so many
    that they are dealt out in turn (3200); captured and replayed."""
    Hk, D, B = 8, 64, 16
    lens = [B * 9 + 1 + i % 40 for i in range(2 * groups)]
    starts, prefix = list(range(0, 2 * groups + 1, 2)), [B * 8] * groups
    c = base._problem(lens, starts, prefix, H, Hk, D, B, BF)
    pkv.set_tuning(shared_prefix=1)
    try:
        want = base._run(c, starts, prefix, BF, max(lens))
        out, q = torch.empty_like(want), c["q"].cuda()
        gs, pl = _ints(starts), _ints(prefix)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_attn_decode_shared(out, q, c["k_pool"], c["v_pool"], c["tables"], c["lens"],
                                         gs, pl, c["scale"], max(lens), 2, B * 8)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    finally:
        pkv.reset_tuning()
    assert pkv.device_errors(clear=True) == 0
    o, bound, _ = ref.decode(c["q"], c["k"], c["v"], c["scale"], BF, once=True)
    ref.check(want, o, bound)

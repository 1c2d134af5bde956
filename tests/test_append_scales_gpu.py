"""8-bit appends against the plain form block by block: where a largest value lies within
fp32's error of a scale's border, either scale will do for that block and head, and its
codes are compared at the one taken; all others, and every value, have to agree."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref
from tests import test_append_rope_gpu as base

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


def _check(pool, scale, start, start_scale, x, err, slots, what):
    got, got_scale = pool.double(), scale.double()
    w_pool, w_scale, bound, doubt = ref.append_q8(start, start_scale, x, err, slots)
    either = {}
    for block, h, other in doubt:
        either.setdefault((block, h), set()).add(other)
    nb, B, Hk, D = start.shape
    free = torch.zeros(nb, Hk, dtype=torch.bool)
    runs = {slots[r[0]] // B: r for r in ref.runs(slots, nb * B, B)[0]}
    for (block, h), others in either.items():
        s = got_scale[block, h].item()
        if s == w_scale[block, h].item():
            continue
        assert s in others, f"{what}: scale {s} of block {block}, head {h}"
        free[block, h] = True
        run = runs[block]
        rows = [slots[t] % B for t in run]
        new, e = x[run][:, h], err[run][:, h]
        # half a step of the value, or of numbers below 2^-6 of the scale
        step = torch.maximum(new.abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10).double())
        assert ((got[block, rows, h] * s - new).abs() <= step * (1 + 2.0 ** -20) + e).all(), what
        if rows[0] > 0:
            kept = ref.round_e4m3(start[block, :rows[0], h] * (start_scale[block, h].item() / s)) \
                if s != start_scale[block, h].item() else start[block, :rows[0], h]
            assert torch.equal(got[block, :rows[0], h], kept), what
        assert torch.equal(got[block, rows[-1] + 1:, h], start[block, rows[-1] + 1:, h]), what
    assert torch.equal(got_scale[~free], w_scale[~free]), f"{what}: scales"
    same = ~free[:, None, :, None].expand_as(got)
    exact = (bound == 0) & same
    assert torch.equal(got[exact].nan_to_num(nan=999.0), w_pool[exact].nan_to_num(nan=999.0)), \
        f"{what}: codes"
    rest = (bound != 0) & same
    off = (got - w_pool).abs() * w_scale[:, None, :, None]
    assert (off <= bound)[rest].all(), f"{what}: values"


def _append(seqs, pad, H, Hk, D, B, rot, inter, dtype, seed):
    torch.cuda.synchronize()
    pkv.device_errors(clear=True)
    gen = torch.Generator().manual_seed(seed)
    slots, pos, blocks = base._slots(seqs, B, gen, pad)
    T, live = len(slots), len(slots) - pad
    _, q, k, v = base._inputs(T, H, Hk, D, dtype, gen)
    table = ref.table64(max(pos[:live]) + 1, rot, dev="cuda")
    k64, k_scale = base._q8_cache(blocks, B, Hk, D, gen)
    v64, v_scale = base._q8_cache(blocks, B, Hk, D, gen, any_scale=True)
    kp, vp, ks, vs = (x.cuda() for x in (k64.to(E4), v64.to(E4), k_scale, v_scale))
    q_out, k_out = (torch.full((T, n, D), 7.0, dtype=dtype, device="cuda") for n in (H, Hk))
    s, p = torch.tensor(slots).cuda(), torch.tensor(pos, dtype=torch.int32)
    pkv.kv_append_rope_q8(kp, vp, ks, vs, k, v, s, p.cuda(), table, q, q_out, k_out, interleaved=inter)
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    zero = torch.zeros(T, Hk, D, dtype=torch.float64)
    _check(vp.cpu(), vs.cpu(), v64, v_scale.double(), v.cpu().double(), zero, slots, "V")
    kr, err = ref.rotate(k.cpu(), table.cpu(), p.clamp(max=table.shape[0] - 1), inter)
    _check(kp.cpu(), ks.cpu(), k64, k_scale.double(), kr, err, slots, "K")
    # the same numbers as the 16-bit append's
    pools = [torch.zeros(blocks, B, Hk, D, dtype=dtype, device="cuda") for _ in range(2)]
    q2, k2 = torch.full_like(q_out, 7.0), torch.full_like(k_out, 7.0)
    pkv.kv_append_rope(*pools, k, v, s, p.cuda(), table, q, q2, k2, interleaved=inter)
    assert torch.equal(q2, q_out) and torch.equal(k2, k_out)


@pytest.mark.parametrize("seqs,pad,H,Hk,D,B,rot,inter,dtype", base.CASES)
@pytest.mark.parametrize("seed", [7, 8])
def test_every_block_and_head(seqs, pad, H, Hk, D, B, rot, inter, dtype, seed):
    _append(seqs, pad, H, Hk, D, B, rot, inter, dtype, seed)


def test_borders_of_the_scale():
    """Largest values that rotation brings to a border exactly: (448, 0) and (0, 448) at
    angles whose cosines round either way, next to ones well apart from it."""
    torch.cuda.synchronize()
    pkv.device_errors(clear=True)
    Hk, D, B, n = 2, 64, 16, 40
    k = torch.zeros(n, Hk, D)
    for t in range(n):
        a = t * 1.0
        for h in range(Hk):
            # the first pair turned back by its angle, so that it comes out near (448, 0)
            k[t, h, 0], k[t, h, D // 2] = 448 * math.cos(a), -448 * math.sin(a)
    k = k.to(torch.float16)
    v = k.clone()
    table = ref.table64(n, D, dev="cuda")
    slots = [t * B + 3 for t in range(n)]
    start = torch.zeros(n, B, Hk, D, dtype=torch.float64)
    scale = torch.full((n, Hk), 0.5, dtype=torch.float64)
    kp, vp = (start.to(E4).cuda() for _ in range(2))
    ks, vs = (scale.float().cuda() for _ in range(2))
    pos = torch.arange(n, dtype=torch.int32)
    pkv.kv_append_rope_q8(kp, vp, ks, vs, k.cuda(), v.cuda(), torch.tensor(slots).cuda(), pos.cuda(), table)
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    kr, err = ref.rotate(k, table.cpu(), pos, False)
    _check(kp.cpu(), ks.cpu(), start, scale, kr, err, slots, "K")
    _check(vp.cpu(), vs.cpu(), start, scale, v.double(), torch.zeros_like(kr), slots, "V")

"""Appends that rotate on the way, into 16-bit and 8-bit pages, against plain
64-bit forms (tests/q8_ref.py, where the tolerances are derived)."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from paged_kv_decode_26_gb300 import _lib
from tests import q8_ref as ref
from tests.cache_ref import EPS

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
E4 = torch.float8_e4m3fn


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


def _slots(seqs, B, gen, pad=0, extra=3):
    """seqs: (tokens before, new tokens).  Slots over a shuffled pool, positions,
    blocks in the pool."""
    pages = [(b % B + n + B - 1) // B for b, n in seqs]
    blocks = sum(pages) + extra
    perm = torch.randperm(blocks, generator=gen).tolist()
    slots, pos = [], []
    for (b, n), c in zip(seqs, pages):
        ids = [perm.pop() for _ in range(c)]
        slots += [ids[(b % B + i) // B] * B + (b + i) % B for i in range(n)]
        pos += range(b, b + n)
    return slots + [-1] * pad, pos + [1 << 30] * pad, blocks


def _inputs(T, H, Hk, D, dtype, gen, fused=True):
    """(qkv on the GPU, its q, k and v views)."""
    qkv = torch.randn(T, H + 2 * Hk, D, generator=gen)
    qkv[:, H:H + Hk] *= (torch.randn(Hk, D, generator=gen) * 1.5).exp()
    qkv = qkv.to(dtype).cuda()
    if fused:
        return qkv, qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    return qkv, *(x.contiguous() for x in (qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]))


CASES = [
    # seqs (before, new), pad, H, Hk, D, B, rot, interleaved, dtype
    ([(0, 1)], 0, 1, 1, 64, 16, 64, False, FP),
    ([(5, 1), (31, 1), (16, 1), (15, 1)], 3, 8, 8, 64, 16, 64, False, BF),
    ([(7, 3), (0, 40), (33, 1)], 1, 8, 2, 128, 32, 128, True, BF),
    ([(100, 17), (3, 29)], 0, 6, 3, 128, 16, 32, False, FP),
    ([(100, 17), (3, 29)], 0, 6, 3, 128, 16, 48, True, FP),
    ([(9, 100)], 5, 24, 12, 64, 32, 16, True, BF),
    ([(i, 1) for i in range(300)], 7, 32, 32, 128, 16, 64, True, BF),
    ([(1000, 700), (3, 600), (0, 33)], 2, 16, 2, 128, 16, 128, False, BF),
    ([(i * 7, 1) for i in range(1100)], 4, 4, 1, 64, 32, 64, False, FP),
]


@pytest.mark.parametrize("seqs,pad,H,Hk,D,B,rot,inter,dtype", CASES)
@pytest.mark.parametrize("with_q", [True, False])
def test_append_rope(seqs, pad, H, Hk, D, B, rot, inter, dtype, with_q):
    _clean()
    gen = torch.Generator().manual_seed(3)
    slots, pos, blocks = _slots(seqs, B, gen, pad)
    T, live = len(slots), len(slots) - pad
    qkv, q, k, v = _inputs(T, H, Hk, D, dtype, gen, fused=with_q)
    table = ref.table64(max(pos[:live]) + 1, rot, dev="cuda")
    kp, vp = (torch.randn(blocks, B, Hk, D, generator=gen).to(dtype).cuda() for _ in range(2))
    k0, v0, qkv0 = kp.clone(), vp.clone(), qkv.clone()
    q_out, k_out = (torch.full((T, n, D), 7.0, dtype=dtype, device="cuda") for n in (H, Hk))
    pkv.kv_append_rope(kp, vp, k, v, torch.tensor(slots).cuda(),
                       torch.tensor(pos, dtype=torch.int32).cuda(), table,
                       q if with_q else None, q_out if with_q else None,
                       k_out if with_q else None, interleaved=inter)
    assert _clean() == 0
    assert torch.equal(qkv, qkv0)
    p = torch.tensor(pos[:live])
    at = torch.tensor(slots[:live])
    want, err = ref.rotate(k[:live].cpu(), table.cpu(), p, inter)
    bound = err + EPS[dtype] / 2 * (want.abs() + err) + (2.0 ** -25 if dtype is FP else 0)
    got = kp.cpu().view(-1, Hk, D)[at].double()
    assert ((got - want).abs() <= bound).all()
    assert torch.equal(got[..., rot:], k[:live].cpu().double()[..., rot:])
    k0.view(-1, Hk, D)[at.cuda()] = kp.view(-1, Hk, D)[at.cuda()]
    assert torch.equal(k0, kp), "rows of no slot changed"
    v0.view(-1, Hk, D)[at.cuda()] = v[:live]
    assert torch.equal(v0, vp)
    if with_q:
        want, err = ref.rotate(q[:live].cpu(), table.cpu(), p, inter)
        bound = err + EPS[dtype] / 2 * (want.abs() + err) + (2.0 ** -25 if dtype is FP else 0)
        assert ((q_out[:live].cpu().double() - want).abs() <= bound).all()
        assert (q_out[live:] == 7.0).all() and (k_out[live:] == 7.0).all()
        assert torch.equal(k_out[:live].cpu(), kp.cpu().view(-1, Hk, D)[at])


def test_append_rope_in_place():
    gen = torch.Generator().manual_seed(4)
    H, Hk, D, B = 8, 2, 128, 16
    slots, pos, blocks = _slots([(3, 50), (0, 9)], B, gen)
    T = len(slots)
    qkv, q, k, v = _inputs(T, H, Hk, D, BF, gen)
    apart = qkv.clone()
    args = (torch.tensor(slots).cuda(), torch.tensor(pos, dtype=torch.int32).cuda(),
            ref.table64(64, 64, dev="cuda"))
    pools = [[torch.zeros(blocks, B, Hk, D, dtype=BF, device="cuda") for _ in range(2)]
             for _ in range(2)]
    q2, k2 = torch.empty(T, H, D, dtype=BF, device="cuda"), torch.empty(T, Hk, D, dtype=BF, device="cuda")
    pkv.kv_append_rope(*pools[0], apart[:, H:H + Hk], apart[:, H + Hk:], *args, apart[:, :H], q2,
                       k2)
    pkv.kv_append_rope(*pools[1], k, v, *args, q, q, k)
    assert _clean() == 0
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, apart[:, H + Hk:])
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])


def test_append_without_rotation_is_kv_append():
    gen = torch.Generator().manual_seed(5)
    Hk, D, B = 4, 64, 16
    slots, _, blocks = _slots([(3, 20), (0, 9)], B, gen, pad=2)
    k, v = (torch.randn(len(slots), Hk, D, generator=gen).to(FP).cuda() for _ in range(2))
    k[0, 0, 0], k[1, 1, 1], v[2, 0, 5] = math.nan, math.inf, -math.inf
    pools = [[torch.zeros(blocks, B, Hk, D, dtype=FP, device="cuda") for _ in range(2)]
             for _ in range(2)]
    s = torch.tensor(slots).cuda()
    pkv.kv_append(*pools[0], k, v, s)
    pkv.kv_append_rope(*pools[1], k, v, s)
    assert _clean() == 0
    for a, b in zip(*pools):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("q8", [False, True])
def test_tokens_outside_the_pool_or_the_table_are_left_out(q8):
    _clean()
    H, Hk, D, B, blocks = 4, 2, 64, 16, 5
    gen = torch.Generator().manual_seed(6)
    slots = [0, 1, blocks * B, 2, 3, 17, -5, 1 << 40]
    pos = [0, 9, 0, 10, -1, 3, 0, 0]
    good = [0, 1, 5]
    qkv, q, k, v = _inputs(len(slots), H, Hk, D, BF, gen)
    table = ref.table64(10, 64, dev="cuda")
    q_out = torch.full((len(slots), H, D), 7.0, dtype=BF, device="cuda")
    kp, vp = (torch.zeros(blocks, B, Hk, D, device="cuda").to(E4 if q8 else BF) for _ in range(2))
    scales = [torch.ones(blocks, Hk, device="cuda") for _ in range(2)] if q8 else []
    fn = pkv.kv_append_rope_q8 if q8 else pkv.kv_append_rope
    fn(kp, vp, *scales, k, v, torch.tensor(slots).cuda(),
       torch.tensor(pos, dtype=torch.int32).cuda(), table, q, q_out)
    assert _clean() == _lib.DEVERR_SLOT | _lib.DEVERR_POSITION
    assert (q_out[[2, 3, 4, 6, 7]] == 7.0).all() and not (q_out[good] == 7.0).all(2).any()
    rows = vp.float().view(-1, Hk, D)
    written = torch.nonzero(rows.abs().amax((1, 2)))[:, 0].tolist()
    assert written == [0, 1, 17]


# ---------------------------------------------------------------- 8-bit pages

def _q8_cache(blocks, B, Hk, D, gen, any_scale=False):
    pool = ref.round_e4m3(torch.randn(blocks, B, Hk, D, generator=gen).double() * 60)
    scale = torch.rand(blocks, Hk, generator=gen) + 0.5 if any_scale else \
        torch.randint(-9, 0, (blocks, Hk), generator=gen).float().exp2()
    return pool, scale


def _check_q8(pool, scale, want, what):
    """Pages against append_q8's (pool, scale, bound, doubt)."""
    w_pool, w_scale, bound, doubt = want
    got, got_scale = pool.double(), scale.double()
    for block, h, other in doubt:
        if got_scale[block, h] == other:
            pytest.skip("a value within fp32's error of a scale's border")
    assert torch.equal(got_scale, w_scale), f"{what}: scales"
    exact = bound == 0
    assert torch.equal(got[exact].nan_to_num(nan=999.0), w_pool[exact].nan_to_num(nan=999.0)), \
        f"{what}: codes"
    off = (got - w_pool).abs() * w_scale[:, None, :, None]
    assert (off <= bound)[~exact].all(), f"{what}: values"
    # and nearly all of them equal: an fp32 error flips few roundings
    if (~exact).sum() > 1000:
        assert (got == w_pool)[~exact].double().mean() > 0.99


@pytest.mark.parametrize("seqs,pad,H,Hk,D,B,rot,inter,dtype", CASES)
@pytest.mark.parametrize("turned", [True, False])
def test_append_rope_q8(seqs, pad, H, Hk, D, B, rot, inter, dtype, turned):
    _clean()
    gen = torch.Generator().manual_seed(7)
    slots, pos, blocks = _slots(seqs, B, gen, pad)
    T, live = len(slots), len(slots) - pad
    qkv, q, k, v = _inputs(T, H, Hk, D, dtype, gen)
    table = ref.table64(max(pos[:live]) + 1, rot, dev="cuda")
    k64, k_scale = _q8_cache(blocks, B, Hk, D, gen)
    v64, v_scale = _q8_cache(blocks, B, Hk, D, gen, any_scale=True)
    kp, vp, ks, vs = (x.cuda() for x in (k64.to(E4), v64.to(E4), k_scale, v_scale))
    q_out, k_out = (torch.full((T, n, D), 7.0, dtype=dtype, device="cuda") for n in (H, Hk))
    s = torch.tensor(slots).cuda()
    p = torch.tensor(pos, dtype=torch.int32)
    zero = torch.zeros(T, Hk, D, dtype=torch.float64)
    if turned:
        pkv.kv_append_rope_q8(kp, vp, ks, vs, k, v, s, p.cuda(), table, q, q_out, k_out,
                              interleaved=inter)
        kr, err = ref.rotate(k.cpu(), table.cpu(), p.clamp(max=table.shape[0] - 1), inter)
    else:
        pkv.kv_append_rope_q8(kp, vp, ks, vs, k, v, s)
        kr, err = k.cpu().double(), zero
    assert _clean() == 0
    _check_q8(vp.cpu(), vs.cpu(), ref.append_q8(v64, v_scale.double(), v.cpu().double(), zero, slots),
              "V")
    _check_q8(kp.cpu(), ks.cpu(), ref.append_q8(k64, k_scale.double(), kr, err, slots), "K")
    if turned:
        # the same numbers as the 16-bit append's
        pools = [torch.zeros(blocks, B, Hk, D, dtype=dtype, device="cuda") for _ in range(2)]
        q2, k2 = torch.full_like(q_out, 7.0), torch.full_like(k_out, 7.0)
        pkv.kv_append_rope(*pools, k, v, s, p.cuda(), table, q, q2, k2, interleaved=inter)
        assert torch.equal(q2, q_out) and torch.equal(k2, k_out)


def test_q8_steps_grow_the_scale():
    """Token after token into the same pages, each larger than what is held."""
    gen = torch.Generator().manual_seed(8)
    Hk, D, B, blocks = 2, 64, 16, 2
    kp, vp = (torch.zeros(blocks, B, Hk, D, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.full((blocks, Hk), math.nan, device="cuda") for _ in range(2))
    pool, scale = torch.zeros(blocks, B, Hk, D, dtype=torch.float64), ks.cpu().double()
    zero = torch.zeros(1, Hk, D, dtype=torch.float64)
    for t in range(20):
        x = (torch.randn(1, Hk, D, generator=gen) * 1.7 ** t).to(BF)
        pkv.kv_append_rope_q8(kp, vp, ks, vs, x.cuda(), x.cuda(), torch.tensor([t]).cuda())
        pool, scale, bound, _ = ref.append_q8(pool, scale, x.double(), zero, [t])
        held = slice(0, t // B + 1)
        assert torch.equal(kp.cpu().double(), pool) and torch.equal(vp.cpu().double(), pool), t
        assert torch.equal(ks.cpu().double()[held], scale[held]), t
    assert _clean() == 0


def test_q8_special_values():
    """NaN stays, infinities saturate, neither sets the scale; zeros; the ends of
    the types; ties; a border of the scale."""
    Hk, D, B = 1, 64, 16
    rows = torch.zeros(9, Hk, D)
    rows[0, 0, :3] = torch.tensor([math.nan, 1.0, -2.0])
    rows[1, 0, :3] = torch.tensor([math.inf, -math.inf, 3.0])
    rows[3, 0, 0] = 448.0                             # exactly the largest
    rows[4, 0, 0] = 450.0                             # bf16's next above
    rows[5, 0, 0] = 3.0e38
    rows[6, 0, 0] = 1.2e-38
    rows[7, 0, :4] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10])   # ties to even
    rows[8, 0, :2] = torch.tensor([math.nan, math.inf])
    rows = rows.to(BF)
    slots = [i * B for i in range(9)]                 # a block each
    kp, vp = (torch.zeros(9, B, Hk, D, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.ones(9, Hk, device="cuda") for _ in range(2))
    pkv.kv_append_rope_q8(kp, vp, ks, vs, rows.cuda(), rows.cuda(), torch.tensor(slots).cuda())
    assert _clean() == 0
    z = torch.zeros(9, Hk, D, dtype=torch.float64)
    want = ref.append_q8(torch.zeros(9, B, Hk, D, dtype=torch.float64),
                         torch.ones(9, Hk, dtype=torch.float64), rows.double(), z, slots)
    # (values below fp32's normal numbers may count as 0, as in all its arithmetic)
    _check_q8(kp.cpu(), ks.cpu(), want, "K")
    _check_q8(vp.cpu(), vs.cpu(), want, "V")
    assert vp[7, 0, 0, 1] == 16.0 and vp[7, 0, 0, 2] == 20.0 and vp[7, 0, 0, 3] == 0.0


@pytest.mark.parametrize("n", [40, 2000])
def test_q8_broken_order(n):
    """Tokens that do not go to rising rows of a block are left out and flagged;
    what stands around them is appended as ever."""
    _clean()
    gen = torch.Generator().manual_seed(9)
    Hk, D, B = 2, 64, 16
    blocks = n // 8 + 4
    order = torch.randperm(blocks, generator=gen).tolist()
    slots = []
    for i in range(n // 10):
        b = order[i] * B
        slots += [b + 3, b + 4, b + 4, b + 9, -1, order[i + 1] * B + 0 if i % 2 else -1,
                  -1, -1, -1, -1] if i % 3 else [b + r for r in range(2, 12)]
    # (a block must not come back: keep the first run of each)
    seen, out, last = set(), [], None
    for s in slots:
        b = s // B if s >= 0 else None
        if b is not None and b != last and b in seen:
            s, b = -1, None
        if b is not None:
            seen.add(b)
        last = b
        out.append(s)
    slots = out
    T = len(slots)
    x = torch.randn(T, Hk, D, generator=gen).to(FP)
    pool, scale = _q8_cache(blocks, B, Hk, D, gen)
    kp, vp, ks, vs = pool.to(E4).cuda(), pool.to(E4).cuda(), scale.cuda(), scale.clone().cuda()
    pkv.kv_append_rope_q8(kp, vp, ks, vs, x.cuda(), x.cuda(), torch.tensor(slots).cuda())
    assert _clean() == _lib.DEVERR_SLOT
    assert ref.runs(slots, blocks * B, B)[1]
    z = torch.zeros(T, Hk, D, dtype=torch.float64)
    want = ref.append_q8(pool, scale.double(), x.double(), z, slots)
    _check_q8(kp.cpu(), ks.cpu(), want, "K")
    _check_q8(vp.cpu(), vs.cpu(), want, "V")


def test_one_slot_for_every_token():
    """The same slot many times: flagged, one of them written."""
    _clean()
    Hk, D, B, T = 2, 128, 32, 1500
    gen = torch.Generator().manual_seed(10)
    x = torch.randn(T, Hk, D, generator=gen).to(BF).cuda()
    kp, vp = (torch.zeros(3, B, Hk, D, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.ones(3, Hk, device="cuda") for _ in range(2))
    pkv.kv_append_rope_q8(kp, vp, ks, vs, x, x, torch.full((T,), B, device="cuda"))
    assert _clean() == _lib.DEVERR_SLOT
    z = torch.zeros(T, Hk, D, dtype=torch.float64)
    want = ref.append_q8(torch.zeros(3, B, Hk, D, dtype=torch.float64),
                         torch.ones(3, Hk, dtype=torch.float64), x.cpu().double(), z, [B] * T)
    _check_q8(kp.cpu(), ks.cpu(), want, "K")


@pytest.mark.parametrize("T", [6, 1200])
def test_on_a_stream_and_in_a_graph(T):
    gen = torch.Generator().manual_seed(11)
    H, Hk, D, B = 8, 2, 64, 16
    slots, pos, blocks = _slots([(5, T)], B, gen)
    qkv, q, k, v = _inputs(T, H, Hk, D, BF, gen)
    s, p = torch.tensor(slots).cuda(), torch.tensor(pos, dtype=torch.int32).cuda()
    table = ref.table64(T + 5, 64, dev="cuda")

    def state():
        return dict(p16=[torch.zeros(blocks, B, Hk, D, dtype=BF, device="cuda") for _ in range(2)],
                    p8=[torch.zeros(blocks, B, Hk, D, device="cuda").to(E4) for _ in range(2)],
                    sc=[torch.full((blocks, Hk), 2.0 ** -9, device="cuda") for _ in range(2)],
                    q=torch.zeros(T, H, D, dtype=BF, device="cuda"))

    def call(st, stream=None):
        pkv.kv_append_rope(*st["p16"], k, v, s, p, table, q, st["q"], stream=stream)
        pkv.kv_append_rope_q8(*st["p8"], *st["sc"], k, v, s, p, table, q, st["q"], stream=stream)

    a, b, c = state(), state(), state()
    call(a)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(b, stream)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    g.replay()
    g.replay()                                # (the same rows again change nothing)
    assert _clean() == 0
    for x in (b, c):
        for key in ("p16", "p8", "sc"):
            for y, z in zip(a[key], x[key]):
                assert torch.equal(y.view(torch.uint8), z.view(torch.uint8)), key
        assert torch.equal(a["q"], x["q"])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [40, 300])
def test_offsets_beyond_32_bits(q8, T):
    """Pools of more than 4 GB and rows 2^24 elements apart, as small ones."""
    gen = torch.Generator().manual_seed(12)
    H, Hk, D, B, stride = 4, 32, 128, 16, 1 << 24
    blocks = -(-T // B) + 1
    nb = (5 << 30) // (B * Hk * D * (1 if q8 else 2))
    _, q, k, v = _inputs(T, H, Hk, D, BF, gen)
    far = [torch.empty(T * stride, dtype=BF, device="cuda") for _ in range(2)]
    kf, qf = (x.as_strided((T, h, D), (stride, D, 1)) for x, h in zip(far, (Hk, H)))
    kf.copy_(k)
    qf.copy_(q)
    pos = torch.arange(3, T + 3, dtype=torch.int32, device="cuda")
    table = ref.table64(T + 3, 128, dev="cuda")

    def call(nb, k, q):
        kind = E4 if q8 else BF
        pools = [torch.empty(nb, B, Hk, D, dtype=kind, device="cuda") for _ in range(2)]
        for p in pools:
            p[-blocks:].view(torch.uint8).zero_()
        sc = [torch.ones(nb, Hk, device="cuda") for _ in range(2)] if q8 else []
        slots = (nb - blocks) * B + 3 + torch.arange(T, device="cuda")
        (pkv.kv_append_rope_q8 if q8 else pkv.kv_append_rope)(*pools, *sc, k, v, slots, pos, table,
                                                              q, q)
        return [p[-blocks:].view(torch.uint8).clone() for p in pools] + [x[-blocks:].clone() for x in sc]

    want = call(blocks, k, q.clone())
    got = call(nb, kf, qf)
    assert _clean() == 0 and want[0].any()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    turned = q.clone()
    pkv.kv_append_rope(torch.empty(1, B, Hk, D, dtype=BF, device="cuda"),
                       torch.empty(1, B, Hk, D, dtype=BF, device="cuda"), k[:B], v[:B],
                       torch.arange(B, device="cuda"), pos[:B], table, turned[:B], turned[:B])
    assert torch.equal(qf[:B], turned[:B])


def test_nothing_to_append():
    k = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    pools = [torch.zeros(2, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2)]
    pkv.kv_append_rope(*pools, k, k, torch.zeros(0, dtype=torch.int64, device="cuda"))
    pools = [x.to(E4) for x in pools]
    sc = [torch.ones(2, 2, device="cuda") for _ in range(2)]
    pkv.kv_append_rope_q8(*pools, *sc, k, k, torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert _clean() == 0


@pytest.mark.parametrize("rot,positions", [(64, 5000), (128, 140000), (16, 1)])
def test_rope_table(rot, positions):
    freq, factor = pkv.rope_frequencies(rot, scaling="yarn", factor=4.0, original_positions=4096)
    t = pkv.rope_table(torch.full((positions, rot), math.nan, device="cuda"), freq, factor)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    want = torch.cat([a.cos(), a.sin()], 1) * torch.tensor(factor, dtype=torch.float32).double()
    # fp32's rounding, and an angle's own in 64 bits (two of them: the product's)
    bound = 2.0 ** -24 * want.abs() + 2 * 2.0 ** -52 * torch.cat([a, a], 1) + 1e-15
    assert ((t.cpu().double() - want).abs() <= bound).all()
    assert _clean() == 0


def test_binding_refusals():
    k = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=BF, device="cuda")
    pools = [torch.zeros(2, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2)]
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    rope = torch.zeros(4, 64, device="cuda")
    for bad in (lambda: pkv.kv_append_rope(*pools, k, k, s.int()),
                lambda: pkv.kv_append_rope(*pools, k, k.half(), s),
                lambda: pkv.kv_append_rope(*pools, k, k, s[:2]),
                lambda: pkv.kv_append_rope(*pools, k, k, s.cpu()),
                lambda: pkv.kv_append_rope(*pools, k.cpu(), k, s),
                lambda: pkv.kv_append_rope(*pools, k, k, s, pos.long(), rope),
                lambda: pkv.kv_append_rope(*pools, k, k, s, pos, rope.half()),
                lambda: pkv.kv_append_rope(*pools, k, k, s, pos, rope, q),
                lambda: pkv.kv_append_rope(*pools, k, k, s, pos, rope, q, q.half()),
                lambda: pkv.kv_append_rope(*pools, k, k, s, pos, rope, q, q[:, :2]),
                lambda: pkv.kv_append_rope(*pools, k.transpose(1, 2), k, s),
                lambda: pkv.kv_append_rope_q8(*pools, *(2 * [torch.ones(2, 2, device="cuda")]), k, k, s),
                lambda: pkv.kv_append_rope_q8(*(x.to(E4) for x in pools),
                                              *(2 * [torch.ones(2, 3, device="cuda")]), k, k, s)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pkv.kv_append_rope(*pools, k, k, s, pos, rope[:, :24].contiguous()),
                lambda: pkv.kv_append_rope(*pools, k, k, s, q=q, q_out=q.clone()),
                lambda: pkv.kv_append_rope(*pools, k, k, s, pos, rope, q, q.clone(), pools[0][0, :3])):
        with pytest.raises(pkv.PagedKVError):
            bad()
    assert _clean() == 0

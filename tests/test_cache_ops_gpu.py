"""The decode that accumulates attention weights and the eviction that goes by
them, against plain 64-bit forms (tests/cache_ref.py, where the tolerances
are derived)."""
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


def _problem(lens, H, Hk, D, B, dtype, seed=1):
    c = ref.paged(lens, B, Hk, D, dtype, seed)
    g = torch.Generator().manual_seed(seed + 100)
    c["q"] = torch.randn(len(lens), H, D, generator=g).to(dtype)
    c["scale"] = 1.0 / math.sqrt(D)
    return c


def _weights(S, cols, seed=5, stride=None):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(S, stride or cols, generator=g).cuda()
    return w[:, :cols]


WEIGHT_CASES = [
    # lens, H, Hk, D, B, dtype, out
    ([1], 1, 1, 64, 16, FP, F32),
    ([0, 1, 15, 16, 17, 0, 33], 8, 8, 128, 16, BF, BF),
    ([200, 3, 77, 0], 8, 8, 64, 16, FP, F32),
    ([31, 32, 33, 500], 8, 2, 128, 32, BF, F32),
    ([1000, 1, 64], 6, 3, 128, 16, BF, BF),          # 3 kv heads: streams of one warp
    ([700, 2], 24, 12, 64, 32, FP, FP),              # 12 kv heads: streams of four
    ([129] * 40 + [0, 5], 16, 2, 64, 16, BF, BF),
    ([5000, 11, 2500], 32, 8, 128, 16, BF, BF),
    ([9000], 8, 1, 128, 32, FP, F32),
    ([7, 300, 0, 0, 45, 1, 1, 1, 90] * 60, 4, 4, 64, 16, BF, F32),   # 540 sequences: scan blocks
    ([300] * 300, 32, 32, 64, 16, FP, FP),
]


@pytest.mark.parametrize("lens,H,Hk,D,B,dtype,out_dtype", WEIGHT_CASES)
def test_decode_weights(lens, H, Hk, D, B, dtype, out_dtype):
    _clean()
    c = _problem(lens, H, Hk, D, B, dtype)
    S, L = len(lens), max(lens)
    w = _weights(S, L + 5, stride=L + 9)
    w0 = w.clone()
    out = torch.full((S, H, D), float("nan"), dtype=out_dtype, device="cuda")
    pkv.paged_attn_decode_weights(out, c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"],
                                  c["lens"], w, c["scale"], L)
    assert _clean() == 0
    o, bound, ws = ref.decode(c["q"], c["k"], c["v"], c["scale"], out_dtype)
    ref.check(out, o, bound, "out")
    for s, n in enumerate(lens):
        want = w0[s, :n].double().cpu() + ws[s][0]
        ref.check(w[s, :n], want, ws[s][1] + 2.0 ** -23 * want, f"weights of {s}")
        assert torch.equal(w[s, n:], w0[s, n:])
        if n:
            assert abs(float((w[s, :n] - w0[s, :n]).double().sum()) - H) < 1e-3 * H


def test_decode_weights_repeats_bit_for_bit_and_accumulates():
    c = _problem([900, 3, 450], 8, 2, 128, 16, BF)
    args = (c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"], c["lens"])
    runs = []
    for _ in range(3):
        w = torch.zeros(3, 900, device="cuda")
        out = torch.empty(3, 8, 128, dtype=BF, device="cuda")
        for _ in range(2):
            pkv.paged_attn_decode_weights(out, *args, w, c["scale"], 900)
        runs.append((out, w))
    for out, w in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(w, runs[0][1])
    assert abs(float(runs[0][1][0].sum()) - 16) < 1e-3


def test_decode_weights_scales():
    """Zero, negative and large scales."""
    for scale in (0.0, -0.1, 4.0):
        c = _problem([100, 17], 4, 2, 64, 16, BF)
        w = torch.zeros(2, 100, device="cuda")
        out = torch.empty(2, 4, 64, dtype=F32, device="cuda")
        pkv.paged_attn_decode_weights(out, c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"],
                                      c["lens"], w, scale, 100)
        o, bound, ws = ref.decode(c["q"], c["k"], c["v"], scale, F32)
        ref.check(out, o, bound, f"scale {scale}")
        for s, n in enumerate([100, 17]):
            ref.check(w[s, :n], ws[s][0], ws[s][1] + 1e-9, f"weights, scale {scale}")


def test_decode_weights_nan_stays_in_its_sequence():
    c = _problem([40, 600, 40], 4, 2, 64, 16, BF)
    slot = int(c["tables"][1, 2])
    c["k_pool"][slot, 3] = float("nan")
    w = torch.zeros(3, 600, device="cuda")
    out = torch.empty(3, 4, 64, dtype=BF, device="cuda")
    pkv.paged_attn_decode_weights(out, c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"],
                                  c["lens"], w, c["scale"], 600)
    assert torch.isnan(out[1]).all() and torch.isnan(w[1]).all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()
    assert torch.isfinite(w[0]).all() and torch.isfinite(w[2]).all()


def test_decode_weights_in_a_graph_and_on_another_stream():
    c = _problem([500, 64, 9], 8, 8, 128, 16, BF)
    q = c["q"].cuda()
    n = pkv.decode_weights_workspace_bytes(3, 8, 8, 128, 16, 500)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    w = torch.zeros(3, 500, device="cuda")
    out = torch.empty(3, 8, 128, dtype=BF, device="cuda")
    call = lambda **kw: pkv.paged_attn_decode_weights(  # noqa: E731
        out, q, c["k_pool"], c["v_pool"], c["tables"], c["lens"], w, c["scale"], 500,
        workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    want, want_w = out.clone(), w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    w.zero_()
    ws.fill_(255)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(w, want_w)
    side = torch.cuda.Stream()
    w.zero_()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    pkv.paged_attn_decode_weights(out, q, c["k_pool"], c["v_pool"], c["tables"], c["lens"], w,
                                  c["scale"], 500, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(w, want_w)


def test_decode_weights_flags_bad_pages_and_lengths():
    _clean()
    c = _problem([64, 40], 4, 4, 64, 16, BF)
    c["tables"][0, 1] = 10 ** 6
    w = torch.zeros(2, 64, device="cuda")
    out = torch.empty(2, 4, 64, dtype=BF, device="cuda")
    pkv.paged_attn_decode_weights(out, c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"],
                                  c["lens"], w, c["scale"], 64)
    assert _clean() == _lib.DEVERR_BLOCK_ID
    assert torch.equal(w[0, 16:32], torch.zeros(16, device="cuda"))
    assert abs(float(w[0].sum()) - 4) < 1e-3
    c = _problem([64, 40], 4, 4, 64, 16, BF)
    c["lens"][1] = -3
    pkv.paged_attn_decode_weights(out, c["q"].cuda(), c["k_pool"], c["v_pool"], c["tables"],
                                  c["lens"], w, c["scale"], 64)
    assert _clean() == _lib.DEVERR_CONTEXT
    assert torch.equal(out[1], torch.zeros_like(out[1]))


# ------------------------------------------------------------------ evict

def _evict_case(lens, keep, recent, Hk, D, B, dtype, weights, new_cols=None, seed=3):
    """Runs kv_evict and checks every output and both pools exactly."""
    _clean()
    S = len(lens)
    pages = [(n + B - 1) // B for n in lens]
    new_pages = (keep + B - 1) // B
    cut = [n > keep for n in lens]
    blocks = sum(pages) + new_pages * sum(cut) + 2
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(blocks, generator=g).tolist()
    tables = torch.full((S, max(pages + [1])), -1, dtype=torch.int32)
    new_tables = torch.full((S, new_pages + 1), -1, dtype=torch.int32)
    for s in range(S):
        for j in range(pages[s]):
            tables[s, j] = perm.pop()
        if cut[s]:
            for j in range(new_pages):
                new_tables[s, j] = perm.pop()
    pools = [torch.randn(blocks, B, Hk, D, generator=g).to(dtype) for _ in range(2)]
    kp, vp = pools[0].cuda(), pools[1].cuda()
    cols = new_cols or keep
    new_w = torch.full((S, cols + 3), 7.0, device="cuda")[:, :cols]
    new_lens = torch.full((S,), -9, dtype=torch.int32, device="cuda")
    kept = torch.full((S, keep), -9, dtype=torch.int32, device="cuda")
    pkv.kv_evict(kp, vp, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 weights.cuda(), new_tables.cuda(), new_lens, new_w, kept, keep, recent)
    assert _clean() == 0
    want = [p.clone() for p in pools]
    for s, n in enumerate(lens):
        idx = ref.evict(weights[s].tolist(), n, keep, recent)
        assert kept[s].tolist() == idx + [-1] * (keep - len(idx))
        assert int(new_lens[s]) == len(idx)
        w = torch.zeros(cols)
        w[:len(idx)] = weights[s][idx]
        assert torch.equal(new_w[s].cpu().view(torch.int32), w.view(torch.int32))
        if cut[s]:
            for j, t in enumerate(idx):
                for i in range(2):
                    want[i][new_tables[s, j // B], j % B] = pools[i][tables[s, t // B], t % B]
    bits = torch.int32 if dtype == F32 else torch.int16
    assert torch.equal(kp.cpu().view(bits), want[0].view(bits))
    assert torch.equal(vp.cpu().view(bits), want[1].view(bits))


def _lognormal(S, cols, seed=11):
    g = torch.Generator().manual_seed(seed)
    return torch.exp(2 * torch.randn(S, cols, generator=g))


@pytest.mark.parametrize("lens,keep,recent,Hk,D,B,dtype", [
    ([1], 1, 0, 1, 64, 16, FP),
    ([2], 1, 1, 1, 64, 16, FP),
    ([2, 0, 1], 1, 0, 8, 64, 16, FP),
    ([200, 3, 64, 65, 0], 64, 16, 8, 64, 16, BF),
    ([77, 500, 33], 33, 33, 2, 128, 32, BF),          # all recent
    ([77, 500, 33], 33, 0, 2, 128, 32, F32),          # none recent
    ([4097, 1023, 1025], 1000, 37, 3, 128, 16, BF),   # odd row width
    ([3000], 2999, 0, 5, 8, 7, FP),                   # odd block size, 80-byte rows
    ([33000, 1], 8191, 511, 1, 64, 16, FP),
    ([130] * 70, 97, 5, 32, 128, 16, BF),             # rows of 8 KB: several parts
])
def test_evict(lens, keep, recent, Hk, D, B, dtype):
    _evict_case(lens, keep, recent, Hk, D, B, dtype, _lognormal(len(lens), max(lens) + 2))


def test_evict_ties_and_special_weights():
    n, inf, nan = 300, math.inf, math.nan
    rows = [
        torch.zeros(n),                                            # all equal
        torch.tensor(([0.0, -0.0] * n)[:n]),                       # the two zeros are equal
        torch.tensor(([nan, 1.0, -inf] * n)[:n]),                  # NaN below -inf
        torch.full((n,), nan),
        torch.tensor(([inf, 1e-40, 2e-40, 0.0] * n)[:n]),          # subnormals keep their order
        torch.tensor(([-1.0, -2.0, 3.0] * n)[:n]),
        torch.arange(n).float(),
        -torch.arange(n).float(),
        torch.tensor([1.0 + 2.0 ** -23 * (i % 5) for i in range(n)]),   # last bits decide
    ]
    w = torch.stack(rows)
    for keep, recent in ((100, 0), (100, 50), (101, 1), (299, 0), (1, 0), (200, 200)):
        _evict_case([n] * len(rows), keep, recent, 2, 64, 16, BF, w, new_cols=keep + 20)


def test_evict_wide_rows_of_weights_and_strides():
    w = _lognormal(3, 900)[:, :700]
    _evict_case([700, 650, 10], 128, 7, 4, 64, 16, BF, w, new_cols=500)


def test_evict_flags_bad_input():
    def call(lens, tables, new_tables, keep=16):
        S = len(lens)
        kp = torch.zeros(8, 16, 2, 64, dtype=BF, device="cuda")
        vp = torch.zeros_like(kp)
        kept = torch.full((S, keep), -9, dtype=torch.int32, device="cuda")
        nl = torch.full((S,), -9, dtype=torch.int32, device="cuda")
        pkv.kv_evict(kp, vp, torch.tensor(tables, dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     torch.rand(S, 64, device="cuda"),
                     torch.tensor(new_tables, dtype=torch.int32, device="cuda"), nl,
                     torch.zeros(S, keep, device="cuda"), kept, keep, 4)
        return _clean(), nl.tolist(), kept
    _clean()
    assert call([40], [[0, 1, 99, -1]], [[5]])[0] == _lib.DEVERR_BLOCK_ID
    assert call([40], [[0, 1, 2, -1]], [[-1]])[0] == _lib.DEVERR_BLOCK_ID
    err, nl, kept = call([65, -1, 20], [[0, 1, 2, 3], [4, 5, 6, 7], [4, 5, -1, -1]],
                         [[5], [6], [7]])
    assert err == _lib.DEVERR_CONTEXT and nl == [0, 0, 16]
    assert (kept[:2] == -1).all()


def test_evict_in_a_graph():
    lens, keep = [200, 90], 64
    w = _lognormal(2, 200).cuda()
    kp = torch.randn(40, 16, 2, 64, device="cuda").to(BF)
    vp = torch.randn(40, 16, 2, 64, device="cuda").to(BF)
    tables = torch.arange(26, dtype=torch.int32, device="cuda").view(2, 13).contiguous()
    new_tables = torch.arange(26, 34, dtype=torch.int32, device="cuda").view(2, 4).contiguous()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = (torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, keep, device="cuda"),
            torch.zeros(2, keep, dtype=torch.int32, device="cuda"))
    call = lambda: pkv.kv_evict(kp, vp, tables, ln, w, new_tables, *outs, keep, 8)  # noqa: E731
    call()
    torch.cuda.synchronize()
    want, pool = [o.clone() for o in outs], kp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for o in outs:
        o.fill_(3)
    kp[26:34] = 0
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs)) and torch.equal(kp, pool)


# ----------------------------------------------- refusals that need a device

def test_workspaces_too_small_or_misaligned_are_refused():
    c = _problem([40, 9], 4, 2, 64, 16, BF)
    q = c["q"].cuda()
    out = torch.full((2, 4, 64), 7.0, dtype=BF, device="cuda")
    w = torch.zeros(2, 40, device="cuda")
    groups = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([0], dtype=torch.int32, device="cuda")
    n_w = pkv.decode_weights_workspace_bytes(2, 4, 2, 64, 16, 40)
    n_s = pkv.decode_shared_workspace_bytes(2, 1, 2, 16, 4, 2, 64, 16, 40)
    buf = torch.empty(max(n_w, n_s) + 512, dtype=torch.uint8, device="cuda")
    for n, call in (
            (n_w, lambda ws: pkv.paged_attn_decode_weights(
                out, q, c["k_pool"], c["v_pool"], c["tables"], c["lens"], w, 0.1, 40,
                workspace=ws)),
            (n_s, lambda ws: pkv.paged_attn_decode_shared(
                out, q, c["k_pool"], c["v_pool"], c["tables"], c["lens"], groups, prefix, 0.1, 40,
                2, 16, workspace=ws))):
        with pytest.raises(pkv.PagedKVError) as e:
            call(buf[:n - 1])
        assert e.value.status == _lib.PKV_ERR_WORKSPACE
        with pytest.raises(pkv.PagedKVError) as e:
            call(buf[16:])
        assert e.value.status == _lib.PKV_ERR_INVALID
        assert (out == 7).all()
        call(buf[:n])
        assert torch.isfinite(out).all() and not (out == 7).all()
        out.fill_(7.0)
    assert _clean() == 0


def test_binding_refuses_bad_tensors():
    c = _problem([40, 9], 4, 2, 64, 16, BF)
    q = c["q"].cuda()
    out = torch.empty(2, 4, 64, dtype=BF, device="cuda")
    ok = dict(out=out, q=q, k_pool=c["k_pool"], v_pool=c["v_pool"], block_tables=c["tables"],
              context_lens=c["lens"], weights=torch.zeros(2, 40, device="cuda"), scale=0.1,
              max_context_len=40)
    for name, bad in (("weights", torch.zeros(2, 39, device="cuda")),
                      ("weights", torch.zeros(3, 40, device="cuda")),
                      ("weights", torch.zeros(2, 40, dtype=torch.float64, device="cuda")),
                      ("weights", torch.zeros(40, 2, device="cuda").t()),
                      ("weights", torch.zeros(1, 40, device="cuda").expand(2, 40)),
                      ("weights", torch.zeros(2, 40)),
                      ("context_lens", c["lens"].long()), ("q", q[:, :, ::2]),
                      ("out", out[:1]), ("v_pool", c["v_pool"].half())):
        with pytest.raises(ValueError):
            pkv.paged_attn_decode_weights(**{**ok, name: bad})


def test_two_streams_at_once():
    """The same call on two streams, a workspace each, interleaved."""
    cases = [_problem([700, 33, 260], 8, 2, 128, 16, BF, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    want, got = [], []
    for c in cases:
        c["qd"] = c["q"].cuda()
        out, w = torch.empty(3, 8, 128, dtype=BF, device="cuda"), torch.zeros(3, 700, device="cuda")
        pkv.paged_attn_decode_weights(out, c["qd"], c["k_pool"], c["v_pool"], c["tables"],
                                      c["lens"], w, c["scale"], 700)
        want.append((out, w))
        got.append((torch.empty_like(out), torch.zeros_like(w)))
    torch.cuda.synchronize()
    for _ in range(20):
        for (out, w), c, s in zip(got, cases, streams):
            with torch.cuda.stream(s):
                w.zero_()
                pkv.paged_attn_decode_weights(out, c["qd"], c["k_pool"], c["v_pool"], c["tables"],
                                              c["lens"], w, c["scale"], 700)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_context_at_all():
    out = torch.full((2, 4, 64), 7.0, dtype=BF, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda").to(BF)
    pool = torch.empty(0, 16, 2, 64, dtype=BF, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    tables = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    pkv.paged_attn_decode_weights(out, q, pool, pool, tables, lens,
                                  torch.zeros(2, 0, device="cuda"), 0.1, 0)
    assert _clean() == 0 and (out == 0).all()
    out.fill_(7.0)
    pkv.paged_attn_decode_shared(out, q, pool, pool, tables, lens, lens[:1], lens[:0], 0.1, 0, 0, 0)
    assert _clean() == 0 and (out == 0).all()


def test_pools_beyond_four_gigabytes():
    """Pages whose byte offsets pass 32 bits: a decode, an accumulation and an
    eviction that reads and writes at both ends of the pool."""
    B, Hk, D, blocks = 32, 16, 128, 36000          # 4.7 GB per pool
    kp = torch.zeros(blocks, B, Hk, D, dtype=BF, device="cuda")
    vp = torch.zeros_like(kp)
    ids = [35999, 0, 35998, 1]
    n = 4 * B - 5
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(4 * B, Hk, D, generator=g).to(BF) for _ in range(2))
    for j, b in enumerate(ids):
        kp[b], vp[b] = k[j * B:(j + 1) * B].cuda(), v[j * B:(j + 1) * B].cuda()
    q = torch.randn(1, 32, D, generator=g).to(BF)
    tables = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty(1, 32, D, dtype=BF, device="cuda")
    w = torch.zeros(1, n, device="cuda")
    scale = 1 / math.sqrt(D)
    pkv.paged_attn_decode_weights(out, q.cuda(), kp, vp, tables, lens, w, scale, n)
    o, bound, ws = ref.decode(q, [k[:n]], [v[:n]], scale, BF)
    ref.check(out, o, bound)
    ref.check(w[0], ws[0][0], ws[0][1] + 1e-7)
    new = torch.tensor([[35997, 2]], dtype=torch.int32, device="cuda")
    nl, kept = torch.zeros_like(lens), torch.zeros(1, 50, dtype=torch.int32, device="cuda")
    pkv.kv_evict(kp, vp, tables, lens, w, new, nl, torch.zeros(1, 50, device="cuda"), kept, 50, 7)
    assert _clean() == 0
    idx = ref.evict(w[0].tolist(), n, 50, 7)
    assert kept[0].tolist() == idx
    got = torch.cat([kp[35997], kp[2]])[:50].cpu()
    assert torch.equal(got, k[idx])
    assert torch.equal(torch.cat([vp[35997], vp[2]])[:50].cpu(), v[idx])


# ------------------------- batches large enough for runs that are taken over

def _large(lens, Hk, D, B, dtype, blocks=400, seed=1):
    """Contexts whose pages are drawn, with repeats, from a small pool."""
    g = torch.Generator().manual_seed(seed)
    width = (max(lens) + B - 1) // B
    tables = torch.randint(blocks, (len(lens), width), generator=g, dtype=torch.int32)
    k, v = (torch.randn(blocks, B, Hk, D, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(len(lens), Hk, D, generator=g).to(dtype)
    return q, k, v, tables


def _large_check(out, w, q, k, v, tables, lens, some, scale, out_dtype):
    for s in some:
        n = lens[s]
        ks, vs = (x[tables[s].long()].flatten(0, 1)[:n] for x in (k, v))
        o, bound, ws = ref.decode(q[s:s + 1], [ks], [vs], scale, out_dtype)
        ref.check(out[s:s + 1], o, bound, f"sequence {s}")
        ref.check(w[s, :n], ws[0][0], ws[0][1] + 2.0 ** -23 * ws[0][0], f"weights of {s}")
        assert (w[s, n:] == 0).all()


@pytest.mark.parametrize("Hk,D,dtype,out_dtype", [(32, 64, BF, BF), (16, 128, FP, F32)])
def test_decode_weights_of_a_large_batch(Hk, D, dtype, out_dtype):
    """128 chunks for every stream and more: a fifth of the work is in short
    runs.  Also captured, and repeated with the same bits."""
    _clean()
    B = 16
    g = torch.Generator().manual_seed(4)
    lens = [1, 0, 17] + torch.randint(1, 6000, (77 * 64 // Hk // 2,), generator=g).tolist() + [6000]
    assert sum((n + 15) // 16 for n in lens) * Hk // 8 >= 152 * 128
    q, k, v, tables = _large(lens, Hk, D, B, dtype)
    scale = 1 / math.sqrt(D)
    S, L = len(lens), max(lens)
    dev = [x.cuda() for x in (q, k, v, tables, torch.tensor(lens, dtype=torch.int32))]
    ws = torch.empty(pkv.decode_weights_workspace_bytes(S, Hk, Hk, D, B, L), dtype=torch.uint8,
                     device="cuda")
    out = torch.full((S, Hk, D), float("nan"), dtype=out_dtype, device="cuda")
    w = torch.zeros(S, L, device="cuda")
    call = lambda: pkv.paged_attn_decode_weights(out, *dev, w, scale, L, workspace=ws)  # noqa: E731
    call()
    assert _clean() == 0
    _large_check(out, w, q, k, v, tables, lens, [0, 1, 2, 3, S // 2, S - 1], scale, out_dtype)
    first, first_w = out.clone(), w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        w.zero_()
        ws.fill_(255)
        graph.replay()
        assert _clean() == 0
        assert torch.equal(out, first) and torch.equal(w, first_w)


def test_decode_weights_short_contexts_under_a_large_bound():
    """The bound asks for runs that can be taken over; the lengths leave them
    empty, or leave whole CTAs without work."""
    B, Hk, D, L = 16, 8, 64, 90000
    for lens in ([40, 0, 1, 900], [0, 0, 0, 0], [5, 0, 0, 0]):
        _clean()
        q, k, v, tables = _large([1000] * 4, Hk, D, B, BF)
        tables = torch.nn.functional.pad(tables, (0, L // B - tables.shape[1]), value=-1)
        out = torch.full((4, Hk, D), float("nan"), dtype=BF, device="cuda")
        w = torch.zeros(4, L, device="cuda")
        pkv.paged_attn_decode_weights(out, q.cuda(), k.cuda(), v.cuda(), tables.cuda(),
                                      torch.tensor(lens, dtype=torch.int32, device="cuda"), w,
                                      0.125, L)
        assert _clean() == 0
        _large_check(out, w, q, k, v, tables[:, :100], lens, range(4), 0.125, BF)

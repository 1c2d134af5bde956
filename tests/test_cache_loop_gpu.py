"""The cache operators together, as a serving loop uses them: prompts
attended straight from the projections, their rows written into pages, decode
steps that share the prompts' common pages, decode steps that accumulate
weights, eviction to a budget, and decode steps on what is left -- every
step's result against a plain 64-bit model of the same loop."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


@pytest.mark.parametrize("H,Hk,D,B,dtype", [(8, 2, 128, 16, torch.bfloat16),
                                            (4, 4, 64, 32, torch.float16)])
def test_serving_loop(H, Hk, D, B, dtype):
    _clean()
    g = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    common, own, steps, keep, recent = 4 * B, [37, 0, 90, 5], 6, 70, 9
    S, G = len(own), H // Hk
    scale = 1 / math.sqrt(D)
    lens = [common + n for n in own]
    blocks = 120
    bm = pkv.BlockManager(blocks, B)
    k_pool = torch.full((blocks, B, Hk, D), float("nan"), dtype=dtype, device="cuda")
    v_pool = k_pool.clone()
    max_blocks = 20
    tables = torch.full((S, max_blocks), -1, dtype=torch.int32)

    # ---- prefill: the common prompt's rows are the same in every sequence
    shared = [rnd(common, Hk, D) for _ in range(2)]
    ks = [torch.cat([shared[0], rnd(n, Hk, D)]) for n in own]
    vs = [torch.cat([shared[1], rnd(n, Hk, D)]) for n in own]
    T = sum(lens)
    q = rnd(T, H, D)
    qkv = torch.cat([q, torch.cat(ks), torch.cat(vs)], 1).cuda()
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    out = torch.empty(T, H, D, dtype=dtype, device="cuda")
    pkv.attn_prompt(out, qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:],
                    torch.tensor(starts, dtype=torch.int32, device="cuda"), scale, max(lens))
    assert _clean() == 0
    for s in range(S):
        n = lens[s]
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        for h in range(H):
            o, _, A, d = ref.attend(q[starts[s]:starts[s + 1], h], ks[s][:, h // G],
                                    vs[s][:, h // G], scale, hidden)
            ref.check(out[starts[s]:starts[s + 1], h], o,
                      ref.out_bound(o, A, d, dtype, dtype, once=True), f"prompt {s}")

    # ---- pages: the common ones once, the others per sequence
    common_ids = [bm.allocate() for _ in range(common // B)]
    slots, rows = [], []
    for s in range(S):
        tables[s, :len(common_ids)] = torch.tensor(common_ids, dtype=torch.int32)
        if s:
            for b in common_ids:
                bm.add_reference(b)
        for j in range(common // B, (lens[s] + B - 1) // B):
            tables[s, j] = bm.allocate()
        for t in range(0 if s == 0 else common, lens[s]):
            slots.append(int(tables[s, t // B]) * B + t % B)
            rows.append(starts[s] + t)
    idx = torch.tensor(rows, device="cuda")
    pkv.kv_append(k_pool, v_pool, qkv[idx, H:H + Hk].contiguous(), qkv[idx, H + Hk:].contiguous(),
                  torch.tensor(slots, dtype=torch.int64, device="cuda"))

    lens_h = torch.tensor(lens, dtype=torch.int32)
    slot_h = torch.empty(S, dtype=torch.int64)
    weights = torch.zeros(S, max_blocks * B, device="cuda")
    model_w = [torch.zeros(max_blocks * B, dtype=torch.float64) for _ in range(S)]

    def step(kind):
        """Append a token per sequence, attend, compare with the model."""
        nonlocal ks, vs
        assert bm.append_slots(tables, lens_h, slot_h) == 0
        k_new, v_new, q1 = rnd(S, Hk, D), rnd(S, Hk, D), rnd(S, H, D)
        pkv.kv_append(k_pool, v_pool, k_new.cuda(), v_new.cuda(), slot_h.cuda())
        ks = [torch.cat([a, b[None]]) for a, b in zip(ks, k_new)]
        vs = [torch.cat([a, b[None]]) for a, b in zip(vs, v_new)]
        o1 = torch.empty(S, H, D, dtype=dtype, device="cuda")
        args = (o1, q1.cuda(), k_pool, v_pool, tables.cuda(), lens_h.cuda())
        L = int(lens_h.max())
        if kind == "shared":
            pkv.paged_attn_decode_shared(
                *args, torch.tensor([0, S], dtype=torch.int32, device="cuda"),
                torch.tensor([common], dtype=torch.int32, device="cuda"), scale, L, S, common)
        elif kind == "weights":
            pkv.paged_attn_decode_weights(*args, weights, scale, L)
        else:
            pkv.paged_attn_decode(*args, scale, L)
        assert _clean() == 0
        o, bound, ws = ref.decode(q1, ks, vs, scale, dtype, once=kind == "shared")
        ref.check(o1, o, bound, kind)
        if kind == "weights":
            for s in range(S):
                model_w[s][:len(ws[s][0])] += ws[s][0]

    for _ in range(steps):
        step("shared")
    for _ in range(steps):
        step("weights")
    # fp32 sums of a few steps: the error stays far below the gaps that decide
    for s in range(S):
        assert torch.allclose(weights[s].double().cpu(), model_w[s], rtol=1e-4, atol=1e-6)

    # ---- cut to the budget; the shared pages live on in the sequences that are not
    before = lens_h.tolist()
    old_tables, old_lens = tables.clone(), lens_h.clone()
    new_tables, old_ids = bm.evict_tables(tables, lens_h, keep)
    new_lens = torch.empty(S, dtype=torch.int32, device="cuda")
    new_w = torch.full_like(weights, -1.0)
    kept = torch.empty(S, keep, dtype=torch.int32, device="cuda")
    pkv.kv_evict(k_pool, v_pool, old_tables.cuda(), old_lens.cuda(), weights, new_tables.cuda(),
                 new_lens, new_w, kept, keep, recent)
    for b in old_ids.tolist():
        bm.free(b)
    assert _clean() == 0
    assert new_lens.tolist() == lens_h.tolist() == [min(n, keep) for n in before]
    # exactly the pages of the new tables are held
    used = {b for row in new_tables.tolist() for b in row if b >= 0}
    assert bm.free_count() == blocks - len(used)
    for s, n in enumerate(before):
        idx = ref.evict(weights[s].tolist(), n, keep, recent)
        assert kept[s].tolist() == idx + [-1] * (keep - len(idx))
        ks[s], vs[s] = ks[s][idx], vs[s][idx]
    tables, weights = new_tables, new_w

    # ---- and on: new tokens land behind the tokens that stayed
    for kind in ("weights", "plain", "weights"):
        step(kind)
    assert [int(n) for n in lens_h] == [min(n, keep) + 3 for n in before]

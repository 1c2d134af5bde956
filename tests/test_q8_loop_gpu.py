"""The rotating appends and the 8-bit attention together, as a serving loop uses
them: prompts chunk by chunk (the first chunk attended straight from the
projections too), decode steps, a fork that copies pages on write, and drafted
tokens to verify -- every result against the plain 64-bit form on the values that
the pages hold, and those against the rotated inputs."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref, q8_ref as ref

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


@pytest.mark.parametrize("H,Hk,D,B,dtype,rot,inter", [
    (8, 4, 128, 16, torch.bfloat16, 128, False), (16, 4, 64, 32, torch.float16, 32, True)])
def test_serving_loop(H, Hk, D, B, dtype, rot, inter):
    _clean()
    gen = torch.Generator().manual_seed(21)
    S, blocks, width, chunk = 3, 60, 12, 48
    G, scale = H // Hk, 1 / math.sqrt(D)
    bm = pkv.BlockManager(blocks, B)
    tables = torch.full((S, width), -1, dtype=torch.int32)
    lens = torch.zeros(S, dtype=torch.int32)
    kp, vp = (torch.full((blocks, B, Hk, D), math.nan, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.full((blocks, Hk), math.nan, device="cuda") for _ in range(2))
    freq, factor = pkv.rope_frequencies(rot, scaling="yarn", factor=4.0, original_positions=64)
    rope = pkv.rope_table(torch.empty(width * B, rot, device="cuda"), freq, factor)
    kept = [[[], []] for _ in range(S)]          # per sequence: rotated keys, values; with errors

    def held(s):
        """The values that sequence s's pages hold, in 64 bits, and their scales."""
        n = int(lens[s])
        t = torch.arange(n)
        b = tables[s].long()[t // B]
        out = []
        for pool, sc in ((kp, ks), (vp, vs)):
            rows = pool.cpu().view(torch.uint8)[b, t % B].view(E4).double()
            out.append((rows * sc.cpu()[b].double()[..., None], sc.cpu()[b].double()[..., None]))
        return out

    def append(counts):
        """New tokens of every sequence; their queries, rotated, and keys."""
        slots, positions = [[] for _ in counts], [[] for _ in counts]
        one = torch.empty(len(counts), dtype=torch.int64)
        for i in range(max(counts)):
            for s, n in enumerate(counts):
                if i >= n:
                    continue
                row, ln = tables[s:s + 1].clone(), lens[s:s + 1].clone()
                st, pairs = bm.append_slots_cow(row, ln, one[:1])
                assert st == 0
                if len(pairs):                  # codes and scales of a shared page
                    dev = pairs.cuda()
                    pkv.swap_blocks_kv(kp, vp, kp, vp, dev)
                    for sc in (ks, vs):
                        pkv.swap_blocks(sc, sc, dev)
                positions[s].append(int(lens[s]))
                tables[s], lens[s] = row[0], ln[0]
                slots[s].append(int(one[0]))
        T = sum(counts)
        qkv = torch.randn(T, H + 2 * Hk, D, generator=gen)
        qkv[:, H:] *= torch.rand(T, 1, 1, generator=gen) * 3 + 0.3     # scales grow and stay
        qkv = qkv.to(dtype).cuda()
        pos = torch.tensor(sum(positions, []), dtype=torch.int32)
        kr, err = ref.rotate(qkv[:, H:H + Hk].cpu(), rope.cpu(), pos, inter)
        q, k = torch.empty_like(qkv[:, :H]), torch.empty_like(qkv[:, H:H + Hk])
        pkv.kv_append_rope_q8(kp, vp, ks, vs, qkv[:, H:H + Hk], qkv[:, H + Hk:],
                              torch.tensor(sum(slots, [])).cuda(), pos.cuda(), rope, qkv[:, :H], q,
                              k, interleaved=inter)
        assert _clean() == 0
        at = 0
        for s, n in enumerate(counts):
            kept[s][0].append((kr[at:at + n], err[at:at + n]))
            v = qkv[at:at + n, H + Hk:].cpu().double()
            kept[s][1].append((v, torch.zeros_like(v)))
            at += n
            for (got, sc), rows in zip(held(s), kept[s]):
                want, e = (torch.cat(x) for x in zip(*rows))
                # half a step of the value, or of numbers below 2^-6 of the scale; and
                # of the smaller scales before
                assert ((got - want).abs() <= want.abs() * 2.0 ** -4 + sc * 2.0 ** -9 + e).all(), s
        return q, k, qkv[:, H + Hk:]

    def check_rows(out, q, counts, once):
        at = 0
        for s, m in enumerate(counts):
            (k, _), (v, _) = held(s)
            n = k.shape[0]
            hidden = torch.ones(m, n, dtype=torch.bool).triu(n - m + 1)
            for h in range(H):
                o, bound = ref.attend_bound(q[at:at + m, h].cpu(), k[:, h // G], v[:, h // G], scale,
                                            dtype, hidden, once=once, chained=True)
                cache_ref.check(out[at:at + m, h], o, bound, f"sequence {s} head {h}")
            at += m

    def attend(counts):
        q, k, v = append(counts)
        start = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        out = torch.empty_like(q)
        pkv.paged_attn_multi_query_q8(out, q, start, kp, vp, ks, vs, tables.cuda(), lens.cuda(),
                                      scale, max(counts), int(lens.max()))
        assert _clean() == 0
        check_rows(out, q, counts, True)
        return q, k, v, start

    # ---- prompts by chunks; the first one from the projections as well
    todo = [70, 33, 101]
    first = True
    while max(todo):
        counts = [min(chunk, n) for n in todo]
        q, k, v, start = attend(counts)
        if first:
            out = torch.empty_like(q)
            pkv.attn_prompt(out, q, k, v, start, scale, max(counts))
            a = 0
            for m in counts:
                hidden = torch.ones(m, m, dtype=torch.bool).triu(1)
                for h in (0, H - 1):
                    o, _, A, d = cache_ref.attend(q[a:a + m, h].cpu(), k[a:a + m, h // G].cpu(),
                                                  v[a:a + m, h // G].cpu(), scale, hidden)
                    cache_ref.check(out[a:a + m, h], o,
                                    cache_ref.out_bound(o, A, d, dtype, dtype, once=True), "prompt")
                a += m
            first = False
        todo = [n - c for n, c in zip(todo, counts)]

    def decode():
        q, _, _ = append([1] * len(lens))
        out = torch.empty_like(q)
        pkv.paged_attn_decode_q8(out, q, kp, vp, ks, vs, tables.cuda(), lens.cuda(), scale,
                                 int(lens.max()))
        assert _clean() == 0
        check_rows(out, q, [1] * len(lens), False)

    for _ in range(5):
        decode()
    # ---- a second answer to sequence 0's prompt: its pages shared, copied on write
    tables = torch.cat([tables, tables[:1]])
    lens = torch.cat([lens, lens[:1]])
    kept.append([list(x) for x in kept[0]])
    for b in tables[0].tolist():
        if b >= 0:
            bm.add_reference(b)
    for _ in range(B + 2):
        decode()
    assert tables[0, 0] == tables[3, 0] and tables[0].tolist() != tables[3].tolist()
    # ---- drafted tokens
    attend([3, 1, 2, 4])

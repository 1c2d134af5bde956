"""Plain 64-bit forms of the rotating appends and of the 8-bit pages.

Errors.  A rotated element a c - b s is formed in fp32 by two roundings, each at
most 2^-24 of |a c| + |b s|: off by `turn_error`.  Stored in 16 bits it is rounded
once more, by half an eps of the type; in e4m3, at scale S, by half a step: 2^-4
of the value, or 2^-10 S below e4m3's normal numbers (2^-6 S).  A block's scale is
a step function of its largest value, so it may be the one of any value within the
error of that.  Without rotation everything is exact.
"""
import math

import torch

E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -117


def table64(positions, rot, stretch=1.0, base=10000.0, dev="cpu"):
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] / stretch * freq
    return torch.cat([a.cos(), a.sin()], 1).float().to(dev)


def rotate(x, table, positions, interleaved):
    """x [T, heads, D] (CPU); table fp32 [P, rot].  float64 (rotated, error of
    its fp32 forming)."""
    x = x.double()
    rot = table.shape[1]
    row = table.double()[positions.long()]
    c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
    out, err = x.clone(), torch.zeros_like(x)
    at = [(2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2) for i in range(rot // 2)]
    a_i, b_i = (torch.tensor(i) for i in zip(*at))
    a, b = x[..., a_i], x[..., b_i]
    out[..., a_i], out[..., b_i] = a * c - b * s, a * s + b * c
    e = 2 * 2.0 ** -24
    err[..., a_i], err[..., b_i] = ((a * c).abs() + (b * s).abs()) * e, \
        ((a * s).abs() + (b * c).abs()) * e
    return out, err


def round_e4m3(x):
    """The nearest number of e4m3 (ties to even, beyond 448: 448, NaN: NaN)."""
    m, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def scale_for(top):
    """The least power of two that brings `top` down to 448."""
    if top <= 0:
        return LEAST_SCALE
    k = math.frexp(top)[1] - 10
    while 2.0 ** k * E4M3_MAX < top:
        k += 1
    return max(2.0 ** k, LEAST_SCALE)


def runs(slots, num_slots, B):
    """The runs of a call by their definition: lists of token indexes that go to
    rising rows of one block, and the tokens that are in none."""
    out, broken, prev = [], [], None
    alive = False
    for t, s in enumerate(slots):
        if not 0 <= s < num_slots:
            prev = None
            continue
        if prev is not None and prev // B == s // B:
            alive = alive and s > prev
            if alive:
                out[-1].append(t)
            else:
                broken.append(t)
        else:
            out.append([t])
            alive = True
        prev = s
    return out, broken


def append_q8(pool, scale, x, err, slots):
    """pool float64 [nb, B, Hk, D] of e4m3 numbers, scale float64 [nb, Hk], x
    float64 [T, Hk, D] with the error of its forming.  Returns (pool, scale,
    largest error of the stored values, list of (block, head, other scale))."""
    nb, B, Hk, D = pool.shape
    pool, scale = pool.clone(), scale.clone()
    doubt = []
    bound = torch.zeros_like(pool)
    for run in runs(slots, nb * B, B)[0]:
        block = slots[run[0]] // B
        rows = [slots[t] % B for t in run]
        new = x[run]
        finite = torch.where(new.isfinite(), new.abs(), torch.zeros_like(new))
        for h in range(Hk):
            top = finite[:, h].max().item()
            off = err[run][:, h].max().item()
            old = scale[block, h].item() if rows[0] > 0 else 0.0
            s = max(scale_for(top), old)
            for other in (scale_for(max(top - off, 0.0)), scale_for(top + off)):
                if max(other, old) != s:
                    doubt.append((block, h, max(other, old)))
            if rows[0] > 0 and s != old:
                kept = pool[block, :rows[0], h] * (old / s)
                pool[block, :rows[0], h] = round_e4m3(kept)
            scale[block, h] = s
            pool[block, rows, h] = round_e4m3(new[:, h] / s)
            bound[block, rows, h] = torch.where(
                err[run][:, h] > 0,
                2 * torch.maximum(new[:, h].abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10)).double()
                + err[run][:, h], torch.zeros_like(err[run][:, h]))
    return pool, scale, bound, doubt


def paged(lens, B, Hk, D, seed, scales="plain", extra_blocks=3):
    """An 8-bit paged cache, poisoned: rows that no context covers are NaN, and so
    are the scales of unused blocks.  scales: "plain" (near 1/200), "wide" (2^-16 ..
    2^8, drawn per block and head), "powers".  Returns dict(k, v: per sequence the
    float64 values [n, Hk, D]; kp, vp, ks, vs, tables, lens on the GPU)."""
    g = torch.Generator().manual_seed(seed)
    pages = [(n + B - 1) // B for n in lens]
    blocks = sum(pages) + extra_blocks
    perm = torch.randperm(blocks, generator=g).tolist()
    tables = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
    out = {}
    for name in ("k", "v"):
        codes = round_e4m3(torch.randn(blocks, B, Hk, D, generator=g).double() * 100)
        if scales == "plain":
            scale = (torch.rand(blocks, Hk, generator=g) + 0.5) / 100
        elif scales == "wide":
            scale = (torch.rand(blocks, Hk, generator=g) * 24 - 16).exp2()
            if name == "k":
                scale = scale.clamp(max=2.0 ** -6)
        else:
            scale = torch.randint(-9, -5, (blocks, Hk), generator=g).float().exp2()
        out[name] = (codes, scale)
    vals = {"k": [], "v": []}
    held = torch.zeros(blocks, B, dtype=torch.bool)
    at = 0
    for s, n in enumerate(lens):
        ids = perm[at:at + pages[s]]
        at += pages[s]
        tables[s, :pages[s]] = torch.tensor(ids, dtype=torch.int32)
        t = torch.arange(n)
        b = torch.tensor(ids + [0])[t // B] if n else torch.zeros(0, dtype=torch.long)
        held[b, t % B] = True
        for name in ("k", "v"):
            codes, scale = out[name]
            vals[name].append(codes[b, t % B] * scale[b].double()[..., None])
    for name in ("k", "v"):
        codes, scale = out[name]
        codes[~held] = math.nan
        scale[~held.any(1)] = math.nan
    return dict(k=vals["k"], v=vals["v"], kp=out["k"][0].to(torch.float8_e4m3fn).cuda(),
                vp=out["v"][0].to(torch.float8_e4m3fn).cuda(), ks=out["k"][1].cuda(),
                vs=out["v"][1].cuda(), tables=tables.cuda(),
                lens=torch.tensor(lens, dtype=torch.int32).cuda())


def attend_bound(q, k, v, scale, out_dtype, hidden=None, once=False, chained=False):
    """64-bit attention of q [R, D] over values k, v [n, D], and the largest error of
    an output element (cache_ref's, with fp16 weights of p b / b_ref: two roundings
    more, and steps of 2^-36 of the largest p b, times codes up to 448; `once`: one
    fp16 part, half an eps of each weight; `chained`: O stays in the tensor core,
    2^-23 of sum p |v| lost per 16 keys)."""
    from tests import cache_ref as ref
    o, p, A, d = ref.attend(q, k, v, scale, hidden)
    if k.shape[0] == 0:
        return o, torch.zeros_like(o)
    bound = ref.out_bound(o, A, d + 2.0 ** -23, torch.float16, out_dtype, once)
    # (paged()'s rows hold codes of 64 and more, so the largest p b is at most 1 / 64
    # of the largest p |v|)
    top = (p * v.abs().amax(-1)).amax(-1)[:, None]
    if chained:
        bound = bound + A * (k.shape[0] / 16 + 1) * 2.0 ** -23
    return o, bound + k.shape[0] * 2.0 ** -36 * E4M3_MAX / 64 * top

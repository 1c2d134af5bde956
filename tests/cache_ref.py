"""Plain 64-bit forms of the cache operators, and how far a kernel may be off.

A kernel's error against the 64-bit form has four sources, each bounded here:

  scores    q . k summed in fp32 over D products: |err| <= D 2^-24 sum |q k|,
            times scale; with the conversion to the log2 domain and the
            subtraction of the maximum, 3 more roundings of |x| <= sum |q k|
            scale.  A softmax weight moves by exp of it: relative
            d = (D + 3) 2^-24 scale max_t sum_d |q_d k_td|, plus 2^-21 for exp2.
  weights   numerator and sum both move by d: 2 d relative, and a sum of n
            positive fp32 terms adds n 2^-24 at most; the pieces' sums are far
            shorter than n, so 2^-18 covers them up to 2^6 terms a chain.
  P V       weights enter the product as hi + lo 16-bit parts (relative
            2^-17 for bf16, 2^-21 for fp16) or, where the operator says so,
            rounded once (half an eps of the type), and n products are summed
            in fp32: 2^-18 as above.  All of it is relative to A = sum p |v|.
  output    half an eps of the output type, relative to the value.
"""
import math

import torch

EPS = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7, torch.float32: 2.0 ** -23}
SPLIT = {torch.float16: 2.0 ** -21, torch.bfloat16: 2.0 ** -17}


def attend(q, k, v, scale, hidden=None):
    """q [R, D], k, v [n, D] in their own types; hidden [R, n] marks masked
    pairs.  Returns float64 (out, p, A = sum p |v|, d) with d [R] the bound of
    a weight's relative error (see above).  n may be 0: zeros."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.zeros(q.shape[0], 0, dtype=torch.float64), z, torch.zeros(q.shape[0])
    x = q @ k.T * scale
    s = q.abs() @ k.abs().T * abs(scale)
    if hidden is not None:
        x = x.masked_fill(hidden, -math.inf)
        s = s.masked_fill(hidden, 0.0)
        v = torch.where(hidden.all(0)[:, None], torch.zeros_like(v), v)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    d = (q.shape[1] + 3) * 2.0 ** -24 * s.amax(-1) + 2.0 ** -21
    return p @ v, p, p @ v.abs(), d


def out_bound(ref, A, d, kv_dtype, out_dtype, once=False):
    """Largest |error| of an output element (shapes [R, D], [R, D], [R])."""
    rounding = EPS[kv_dtype] / 2 if once else SPLIT[kv_dtype]
    inner = A * (2 * d[:, None] + 2.0 ** -17 + rounding)
    return inner + EPS[out_dtype] / 2 * (ref.abs() + inner) + 1e-30


def weight_bound(p, d):
    """Largest |error| of sum_h p[h, t] (p [H, n], d [H])."""
    return (p * (2 * d[:, None] + 2.0 ** -18)).sum(0) + p.sum(0) * p.shape[0] * 2.0 ** -24


def paged(lens, B, Hk, D, dtype, seed, shared=None, extra_blocks=3, dev="cuda"):
    """A poisoned paged cache: rows that no context covers are NaN.  shared:
    (group starts, prefix tokens per group): members longer than the prefix
    point at the group's pages.  Returns dict(k, v: per sequence [n, Hk, D]
    on the CPU, k_pool, v_pool, tables, lens on `dev`)."""
    g = torch.Generator().manual_seed(seed)
    pages = [(n + B - 1) // B for n in lens]
    width = max(pages + [1])
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    ks = [torch.randn(n, Hk, D, generator=g).to(dtype) for n in lens]
    vs = [torch.randn(n, Hk, D, generator=g).to(dtype) for n in lens]
    owner = {}
    if shared is not None:
        for gi, (a, b) in enumerate(zip(shared[0], shared[0][1:])):
            pl = shared[1][gi]
            first = None
            for s in range(a, b):
                if lens[s] < pl:
                    continue
                if first is None:
                    first = s
                ks[s][:pl], vs[s][:pl] = ks[first][:pl], vs[first][:pl]
                for j in range(pl // B):
                    owner[(s, j)] = (first, j)
    need = sum(1 for s in range(len(lens)) for j in range(pages[s])
               if owner.get((s, j), (s, j)) == (s, j))
    blocks = need + extra_blocks
    perm = torch.randperm(blocks, generator=g).tolist()
    k_pool = torch.full((blocks, B, Hk, D), float("nan"), dtype=dtype)
    v_pool = k_pool.clone()
    at = {}
    for s in range(len(lens)):
        for j in range(pages[s]):
            key = owner.get((s, j), (s, j))
            if key not in at:
                at[key] = perm.pop()
                rows = min(B, lens[s] - j * B)
                k_pool[at[key], :rows] = ks[s][j * B:j * B + rows]
                v_pool[at[key], :rows] = vs[s][j * B:j * B + rows]
            tables[s, j] = at[key]
    return dict(k=ks, v=vs, k_pool=k_pool.to(dev), v_pool=v_pool.to(dev), tables=tables.to(dev),
                lens=torch.tensor(lens, dtype=torch.int32, device=dev), free=perm)


def decode(q, ks, vs, scale, out_dtype, once=False):
    """Per sequence paged decode.  q [S, H, D] (CPU).  Returns (out, bound)
    [S, H, D], and per sequence (weights, bound) [n]."""
    S, H, D = q.shape
    out = torch.zeros(S, H, D, dtype=torch.float64)
    bound = torch.zeros_like(out)
    weights = []
    for s in range(S):
        Hk = ks[s].shape[1]
        G = H // Hk
        w = torch.zeros(ks[s].shape[0], dtype=torch.float64)
        wb = torch.zeros_like(w)
        for j in range(Hk):
            o, p, A, d = attend(q[s, j * G:(j + 1) * G], ks[s][:, j], vs[s][:, j], scale)
            out[s, j * G:(j + 1) * G] = o
            bound[s, j * G:(j + 1) * G] = out_bound(o, A, d, ks[s].dtype, out_dtype, once)
            if p.shape[1]:
                w += p.sum(0)
                wb += weight_bound(p, d)
        weights.append((w, wb))
    return out, bound, weights


def evict(weights, n, keep, recent):
    """Indexes that stay, by the definition (weights: list of floats)."""
    if n <= keep:
        return list(range(n))
    key = [(-math.inf if math.isnan(w) else w, math.isnan(w)) for w in weights[:n]]
    old = sorted(range(n - recent), key=lambda t: (-key[t][0], key[t][1], t))
    return sorted(old[:keep - recent]) + list(range(n - recent, n))


def check(got, ref, bound, what=""):
    g = got.detach().double().cpu()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    err = (g - ref).abs()
    worst = (err / bound.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} of the bound (max |err| {err.max():.3g})"

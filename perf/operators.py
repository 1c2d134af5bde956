"""What the cache's prompt, prefix-sharing and eviction operators are measured on.

Four operators of the paged KV cache:

  prompt   causal attention over whole packed prompts (attn_prompt): the
           prefill of new requests, straight from the projections' output
  shared   a decode step of sequences that share long prefixes, each prefix
           attended once for its group (paged_attn_decode_shared)
  weights  a decode step that adds every cached token's attention weight to a
           running sum (paged_attn_decode_weights)
  evict    a cache cut to a budget: the last tokens and the heaviest earlier
           ones stay, compacted into new pages (kv_evict)

`run` computes them by elementary torch operations in fp32, or, with `own`,
by the library's calls.  Lengths follow from the case alone (so `work` can
count them), values and page placement from the seed.
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a handful of short prompts on a small model: latency counts
        dict(name="prompt_tiny", op="prompt", S=4, H=8, Hk=8, D=64, lo=1, hi=200, dtype="fp16",
             out="fp16"),
        # a prefill batch of grouped-query heads, prompts of mixed lengths
        dict(name="prompt_packed_gqa", op="prompt", S=16, H=32, Hk=8, D=128, lo=128, hi=2048,
             dtype="bf16", out="bf16"),
        # long documents, one kv head per query head
        dict(name="prompt_long_mha", op="prompt", S=2, H=32, Hk=32, D=128, lo=4096, hi=8192,
             dtype="bf16", out="bf16"),
        # a few samples of one short prompt, fp32 result
        dict(name="shared_tiny", op="shared", S=4, groups=1, prefix=64, H=8, Hk=8, D=64, B=16,
             lo=1, hi=100, dtype="fp16", out="fp32"),
        # sixteen templates, eight requests each: 64 shared pages a group
        dict(name="shared_groups_gqa", op="shared", S=128, groups=16, prefix=1024, H=32, Hk=8,
             D=128, B=16, lo=16, hi=4096, dtype="bf16", out="bf16"),
        # one long system prompt or document under every request of the batch
        dict(name="shared_document", op="shared", S=256, groups=1, prefix=16384, H=32, Hk=8,
             D=128, B=16, lo=16, hi=1024, dtype="bf16", out="bf16"),
        # the small model's decode step, fp32 result
        dict(name="weights_tiny", op="weights", S=4, H=8, Hk=8, D=64, B=16, lo=1, hi=200,
             dtype="fp16", out="fp32"),
        # a serving batch with one kv head per query head
        dict(name="weights_mha", op="weights", S=64, H=32, Hk=32, D=128, B=16, lo=512, hi=4096,
             dtype="bf16", out="bf16"),
        # a few long contexts, grouped-query heads, larger pages
        dict(name="weights_long_gqa", op="weights", S=8, H=32, Hk=8, D=128, B=32, lo=8192,
             hi=32768, dtype="bf16", out="bf16"),
        # the small model's cache cut to 64 tokens a sequence
        dict(name="evict_tiny", op="evict", S=4, Hk=8, D=64, B=16, lo=1, hi=200, keep=64,
             recent=16, dtype="fp16"),
        # a serving batch cut to 1024 tokens a sequence
        dict(name="evict_mha", op="evict", S=64, Hk=32, D=128, B=16, lo=512, hi=4096, keep=1024,
             recent=256, dtype="bf16"),
        # long contexts cut to a quarter
        dict(name="evict_long_gqa", op="evict", S=4, Hk=8, D=128, B=32, lo=32768, hi=32768,
             keep=8192, recent=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prompt", "shared", "weights", "evict"])
    Hk = rng.choice([1, 2, 4, 8, 16, 32])
    G = rng.choice([g for g in (1, 2, 4, 8) if g * Hk <= 64])
    D = rng.choice([64, 128])
    B = rng.choice([16, 32])
    dt = rng.choice(["bf16", "fp16"])
    if op == "prompt":
        hi = _log(rng, 2, min(8192, math.isqrt(25 * 10 ** 8 // (G * Hk))))
        S = _log(rng, 1, min(64, 25 * 10 ** 8 // (G * Hk * hi * hi)))
        return dict(op=op, S=S, H=G * Hk, Hk=Hk, D=D, lo=_log(rng, 1, hi), hi=hi, dtype=dt,
                    out=rng.choice([dt, dt, "fp32"]))
    if op == "shared":
        prefix = B * _log(rng, 1, 16384 // B)
        hi = _log(rng, 1, 4096)
        S = _log(rng, 1, max(1, min(256, 4 * 10 ** 9 // (Hk * D * (prefix + hi)),
                                    15 * 10 ** 7 // (Hk * D * hi))))
        groups = _log(rng, 1, max(1, min(S, 15 * 10 ** 7 // (Hk * D * prefix))))
        return dict(op=op, S=S, groups=groups, prefix=prefix, H=G * Hk, Hk=Hk, D=D, B=B,
                    lo=_log(rng, 1, hi), hi=hi, dtype=dt, out=rng.choice([dt, dt, "fp32"]))
    hi = _log(rng, 1, 32768)
    S = _log(rng, 1, max(1, min(256, (5 * 10 ** 8 if op == "weights" else 22 * 10 ** 7)
                            // (Hk * D * hi))))
    lo = _log(rng, 1, hi)
    if op == "weights":
        return dict(op=op, S=S, H=G * Hk, Hk=Hk, D=D, B=B, lo=lo, hi=hi, dtype=dt,
                    out=rng.choice([dt, dt, "fp32"]))
    keep = _log(rng, 1, hi)
    return dict(op=op, S=S, Hk=Hk, D=D, B=B, lo=lo, hi=hi, keep=keep,
                recent=rng.randint(0, keep), dtype=dt)


def _lens(case):
    """The sequences' lengths (behind the shared prefix, where there is one),
    from the case alone.  The longest is the upper end of the range."""
    r = random.Random("%(op)s %(S)d %(lo)d %(hi)d" % case)
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]
    n[r.randrange(case["S"])] = case["hi"]
    return n


def _groups(case):
    """Sequences 0 .. S-1 cut into `groups` runs of nearly equal size."""
    S, g = case["S"], case["groups"]
    return [S * i // g for i in range(g + 1)]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _tables(gen, lens, B, spare=0, shared=None):
    """Page tables of sequences of these lengths over a shuffled pool with
    `spare` more blocks; shared: (group starts, pages that a group shares).
    Returns (tables [S, pages], spare ids, blocks in the pool)."""
    pages = [(n + B - 1) // B for n in lens]
    width = max(max(pages), 1)
    first = [0] * len(lens)
    if shared is not None:
        starts, common = shared
        at = [s for a, b in zip(starts, starts[1:]) for s in [a] * (b - a)]
        first = [common] * len(lens)
        n_common = common * (len(starts) - 1)
    else:
        n_common = 0
    used = n_common + sum(p - f for p, f in zip(pages, first))
    total = used + spare
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    t = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")[None, :]
    n_pages, head = _ints(pages)[:, None], _ints(first)[:, None]
    own_pages = (col >= head) & (col < n_pages)
    t[own_pages] = perm[n_common:used]
    if shared is not None:
        group = {a: i for i, a in enumerate(dict.fromkeys(at))}
        row = _ints([group[a] for a in at], torch.int64)
        t[:, :common] = perm[:n_common].view(-1, common)[row]
    return t.contiguous(), perm[used:], total


def _pools(gen, blocks, case, dt):
    shape = (blocks, case["B"], case["Hk"], case["D"])
    return tuple(torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in range(2))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    lens = _lens(case)
    S, Hk, D = case["S"], case["Hk"], case["D"]
    st = dict(op=case["op"], case=dict(case), scale=1.0 / math.sqrt(D))
    if case["op"] == "prompt":
        H, T = case["H"], sum(lens)
        # the fused projection's output; q, k and v are views of it
        qkv = torch.randn((T, H + 2 * Hk, D), generator=gen, device="cuda", dtype=dt)
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        st.update(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], q_start=_ints(starts),
                  max_len=max(lens),
                  out=torch.zeros((T, H, D), device="cuda", dtype=_TYPES[case["out"]]))
        return st
    B = case["B"]
    if case["op"] == "evict":
        keep = case["keep"]
        new_pages = (keep + B - 1) // B
        evicted = [n > keep for n in lens]
        tables, spare, blocks = _tables(gen, lens, B, spare=new_pages * sum(evicted))
        new_tables = torch.full((S, new_pages), -1, dtype=torch.int32, device="cuda")
        shared_width = min(new_pages, tables.shape[1])
        new_tables[:, :shared_width] = tables[:, :shared_width]
        new_tables[_ints(evicted, torch.bool)] = spare.view(-1, new_pages)
        k_pool, v_pool = _pools(gen, blocks, case, dt)
        # accumulated softmax weights: a few heavy tokens, many light ones,
        # and the newest ones not yet attended to
        weights = torch.randn((S, max(lens)), generator=gen, device="cuda").mul_(2.0).exp_()
        weights[torch.rand((S, max(lens)), generator=gen, device="cuda") < 0.02] = 0.0
        st.update(k_pool=k_pool, v_pool=v_pool, tables=tables, lens=_ints(lens), weights=weights,
                  new_tables=new_tables,
                  new_lens=torch.zeros(S, dtype=torch.int32, device="cuda"),
                  new_weights=torch.zeros((S, keep), device="cuda"),
                  kept=torch.zeros((S, keep), dtype=torch.int32, device="cuda"),
                  keep=keep, recent=case["recent"])
        return st
    H = case["H"]
    if case["op"] == "shared":
        starts = _groups(case)
        lens = [case["prefix"] + n for n in lens]
        tables, _, blocks = _tables(gen, lens, B, shared=(starts, case["prefix"] // B))
        st.update(group_start=_ints(starts),
                  prefix_lens=_ints([case["prefix"]] * case["groups"]),
                  max_group=max(b - a for a, b in zip(starts, starts[1:])),
                  max_prefix=case["prefix"])
    else:
        tables, _, blocks = _tables(gen, lens, B)
        # what a step or so of H heads has left on each token
        st.update(weights=torch.rand((S, max(lens)), generator=gen, device="cuda")
                  .mul_(H / max(lens)))
    k_pool, v_pool = _pools(gen, blocks, case, dt)
    st.update(q=torch.randn((S, H, D), generator=gen, device="cuda", dtype=dt), k_pool=k_pool,
              v_pool=v_pool, tables=tables, lens=_ints(lens), max_len=max(lens),
              out=torch.zeros((S, H, D), device="cuda", dtype=_TYPES[case["out"]]))
    return st


# ------------------------------------------------------------ plain forms

def _slots(tables, B, width):
    """Pool row of logical token 0 .. width-1 of every sequence; an unused
    table entry gives some valid row."""
    t = torch.arange(width, device=tables.device)
    return tables.long().clamp(min=0)[:, t // B] * B + t % B


def _plain_prompt(st):
    q, k, v, starts, L = st["q"], st["k"], st["v"], st["q_start"].long(), st["max_len"]
    T, H, D = q.shape
    G = H // k.shape[1]
    pos = torch.arange(L, device=q.device)
    at = (starts[:-1, None] + pos).clamp(max=T - 1)              # [S, L] rows, padded
    qf = q.float()[at].transpose(1, 2)                            # [S, H, L, D]
    kf = k.float()[at].transpose(1, 2).repeat_interleave(G, 1)
    vf = v.float()[at].transpose(1, 2).repeat_interleave(G, 1)
    x = torch.matmul(qf, kf.transpose(2, 3)).mul_(st["scale"])
    x.masked_fill_(pos[None, :] > pos[:, None], float("-inf"))
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    o = torch.matmul(x, vf).transpose(1, 2)                       # [S, L, H, D]
    t = torch.arange(T, device=q.device)
    s = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    st["out"].copy_(o[s, t - starts[s]])
    return st["out"]


def _plain_decode(st):
    """(out in fp32, softmax weights [S, H, L])."""
    q, L, lens = st["q"], st["max_len"], st["lens"]
    S, H, D = q.shape
    B, Hk = st["k_pool"].shape[1:3]
    rows = _slots(st["tables"], B, L)
    k = st["k_pool"].view(-1, Hk, D)[rows].float().transpose(1, 2)    # [S, Hk, L, D]
    x = torch.matmul(q.float().view(S, Hk, H // Hk, D), k.transpose(2, 3)).mul_(st["scale"])
    del k
    x.masked_fill_((torch.arange(L, device=q.device) >= lens[:, None])[:, None, None], float("-inf"))
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    v = st["v_pool"].view(-1, Hk, D)[rows].float().transpose(1, 2)
    return torch.matmul(x, v).reshape(S, H, D), x.reshape(S, H, L)


def _plain_evict(st):
    w, n, keep, recent = st["weights"], st["lens"][:, None], st["keep"], st["recent"]
    S, L = w.shape
    B = st["k_pool"].shape[1]
    t = torch.arange(L, device=w.device)[None, :]
    # the newest tokens come first, then by weight (the lower index of equal ones)
    rank = torch.where(t < n - recent, w, torch.where(t < n, math.inf, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[1]), value=L)
    j = torch.arange(keep, device=w.device)[None, :]
    cut = n > keep
    kept = torch.where(cut, torch.sort(order, dim=1).values, j)
    src_at = torch.minimum(kept, n - 1).long()
    st["kept"].copy_(torch.where(j < n, kept, -1))
    st["new_lens"].copy_(n[:, 0].clamp(max=keep))
    st["new_weights"].copy_(torch.where(j < n, w.gather(1, src_at), 0.0))
    src = _slots(st["tables"], B, L).gather(1, src_at)
    dst = torch.where(cut, _slots(st["new_tables"], B, keep), src)
    for pool in (st["k_pool"], st["v_pool"]):
        rows = pool.view(-1, pool.shape[2] * pool.shape[3])
        rows[dst.reshape(-1)] = rows[src.reshape(-1)]


def run(st):
    if own:
        import paged_kv_decode_26_gb300 as pkv
    if st["op"] == "prompt":
        if own:
            pkv.attn_prompt(st["out"], st["q"], st["k"], st["v"], st["q_start"], st["scale"],
                            st["max_len"])
        else:
            _plain_prompt(st)
        return st["out"]
    if st["op"] == "shared":
        if own:
            pkv.paged_attn_decode_shared(st["out"], st["q"], st["k_pool"], st["v_pool"],
                                         st["tables"], st["lens"], st["group_start"],
                                         st["prefix_lens"], st["scale"], st["max_len"],
                                         st["max_group"], st["max_prefix"])
        else:
            st["out"].copy_(_plain_decode(st)[0])
        return st["out"]
    if st["op"] == "weights":
        if own:
            pkv.paged_attn_decode_weights(st["out"], st["q"], st["k_pool"], st["v_pool"],
                                          st["tables"], st["lens"], st["weights"], st["scale"],
                                          st["max_len"])
        else:
            o, p = _plain_decode(st)
            st["out"].copy_(o)
            st["weights"].add_(p.sum(1))
        return {"out": st["out"], "weights": st["weights"]}
    if own:
        pkv.kv_evict(st["k_pool"], st["v_pool"], st["tables"], st["lens"], st["weights"],
                     st["new_tables"], st["new_lens"], st["new_weights"], st["kept"], st["keep"],
                     st["recent"])
    else:
        _plain_evict(st)
    return {k: st[k] for k in ("k_pool", "v_pool", "new_lens", "new_weights", "kept")}


# ----------------------------------------------------------- 64-bit values

def _softmax64(x):
    e = torch.exp(x - x.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def exact(case, seed):
    st = prepare(case, seed)
    lens = _lens(case)
    if case["op"] == "prompt":
        G = case["H"] // case["Hk"]
        out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for n in lens:
            hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            for h in range(case["H"]):
                q, k, v = (a[at:at + n, i].double() for a, i in
                           ((st["q"], h), (st["k"], h // G), (st["v"], h // G)))
                p = _softmax64((q @ k.T * st["scale"]).masked_fill(hidden, -math.inf))
                out[at:at + n, h] = p @ v
            at += n
        return out
    B, Hk = case["B"], case["Hk"]
    rows = [torch.cat([torch.arange(b * B, b * B + B) for b in t if b >= 0])
            for t in st["tables"].tolist()]
    if case["op"] == "evict":
        k, v = st["k_pool"].view(-1, Hk * case["D"]), st["v_pool"].view(-1, Hk * case["D"])
        weights = st["weights"].tolist()
        new_tables = st["new_tables"].tolist()
        src, dst = [], []
        for s, n in enumerate(lens):
            old = n - case["recent"]
            kept = list(range(n))
            if n > case["keep"]:
                heavy = sorted(range(old), key=lambda t: (-weights[s][t], t))
                kept = sorted(heavy[:case["keep"] - case["recent"]]) + list(range(max(old, 0), n))
                src += [int(rows[s][t]) for t in kept]
                dst += [new_tables[s][j // B] * B + j % B for j in range(len(kept))]
            st["kept"][s] = _ints(kept + [-1] * (case["keep"] - len(kept)))
            st["new_lens"][s] = len(kept)
            st["new_weights"][s] = 0.0
            st["new_weights"][s, :len(kept)] = st["weights"][s][_ints(kept, torch.int64)]
        for pool in (k, v):
            pool[_ints(dst, torch.int64)] = pool[_ints(src, torch.int64)]
        return {"k_pool": st["k_pool"].double(), "v_pool": st["v_pool"].double(),
                "new_lens": None, "new_weights": st["new_weights"].double(), "kept": None}
    S, H, D = st["q"].shape
    out = torch.empty((S, H, D), dtype=torch.float64, device="cuda")
    for s in range(S):
        n = int(st["lens"][s])
        r = rows[s][:n].cuda()
        k, v = (p.view(-1, Hk, D)[r].double().permute(1, 0, 2) for p in (st["k_pool"], st["v_pool"]))
        p = _softmax64(st["q"][s].double().view(Hk, H // Hk, D) @ k.transpose(1, 2) * st["scale"])
        out[s] = (p @ v).view(H, D)
        if case["op"] == "weights":
            st["weights"] = st["weights"].double()
            st["weights"][s, :n] += p.sum((0, 1))
    return {"out": out, "weights": st["weights"]} if case["op"] == "weights" else out


# ------------------------------------------------------------ what it costs

def work(case):
    """Each input that the operator needs read once, each output written
    once; products and exponentials are counted as the two matrix products."""
    lens = _lens(case)
    S, Hk, D = case["S"], case["Hk"], case["D"]
    e = 2
    if case["op"] == "evict":
        moved = sum(case["keep"] for n in lens if n > case["keep"])
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": 2 * 2 * moved * Hk * D * e + 4 * sum(lens) + (4 + 4) * S * case["keep"]
                + 4 * 2 * S, "flops": kept}
    H = case["H"]
    eo = 4 if case["out"] == "fp32" else 2
    if case["op"] == "prompt":
        T = sum(lens)
        return {"bytes": T * D * ((H + 2 * Hk) * e + H * eo) + 4 * (S + 1),
                "flops": 4 * H * D * sum(n * (n + 1) // 2 for n in lens)}
    small = S * H * D * (e + eo) + 4 * S
    if case["op"] == "shared":
        B = case["B"]
        tokens = sum(lens) + case["groups"] * case["prefix"]
        pages = sum((n + B - 1) // B for n in lens) + case["groups"] * case["prefix"] // B
        return {"bytes": 2 * tokens * Hk * D * e + 4 * pages + 8 * case["groups"] + small,
                "flops": 4 * H * D * (sum(lens) + S * case["prefix"])}
    tokens = sum(lens)
    pages = sum((n + case["B"] - 1) // case["B"] for n in lens)
    return {"bytes": 2 * tokens * Hk * D * e + 4 * pages + 2 * 4 * tokens + small,
            "flops": 4 * H * D * tokens}

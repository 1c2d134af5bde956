"""What the cache's rotating appends and its 8-bit form are measured on.

Four operators of the paged KV cache:

  append     new tokens into the 16-bit pages, keys and queries rotated by
             their positions on the way (kv_append_rope)
  append_q8  the same into pages of 8 bits (e4m3) with a scale for each block
             and kv head, which grows with what the block holds
             (kv_append_rope_q8)
  decode_q8  a decode step over 8-bit pages (paged_attn_decode_q8)
  chunk_q8   causal attention of a chunk of new tokens per sequence over 8-bit
             pages (paged_attn_multi_query_q8)

`run` computes them by elementary torch operations in fp32, or, with `own`, by
the library's calls.  Lengths follow from the case alone (so `work` can count
them), values and page placement from the seed.  A rotation table holds, for
every position, the cosines of its angles and then their sines.
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_E4M3_MAX = 448.0
_LEAST_SCALE = 2.0 ** -117      # of a block whose rows are all zero


def listed():
    return [
        # one decode step of a handful of requests to a small model: latency
        dict(name="append_tiny", op="append", S=4, lo=1, hi=1, before=200, pad=0, H=8, Hk=8, D=64,
             B=16, rot=64, interleaved=False, stretch=1.0, dtype="fp16"),
        # a large decode batch, one kv head per query head, half of the head
        # rotated in neighbouring pairs, padded to a captured batch size
        dict(name="append_batch_partial", op="append", S=250, lo=1, hi=1, before=4096, pad=6, H=32,
             Hk=32, D=128, B=16, rot=64, interleaved=True, stretch=1.0, dtype="bf16"),
        # a prefill batch of grouped-query heads behind cached prefixes,
        # positions stretched for a longer context
        dict(name="append_prefill_gqa", op="append", S=16, lo=128, hi=2048, before=16384, pad=0,
             H=32, Hk=8, D=128, B=16, rot=128, interleaved=False, stretch=4.0, dtype="bf16"),
        # a few tokens to verify per request of a small model, pages partly filled
        dict(name="append_q8_tiny", op="append_q8", S=4, lo=1, hi=4, before=200, pad=0, H=8, Hk=8,
             D=64, B=16, rot=64, interleaved=False, stretch=1.0, dtype="fp16"),
        # a large decode batch: every block holds tokens, whose scale may grow
        dict(name="append_q8_batch", op="append_q8", S=256, lo=1, hi=1, before=8192, pad=0, H=32,
             Hk=8, D=128, B=16, rot=128, interleaved=False, stretch=1.0, dtype="bf16"),
        # a prefill batch, one kv head per query head, larger pages
        dict(name="append_q8_prefill_mha", op="append_q8", S=8, lo=300, hi=2048, before=4096,
             pad=0, H=32, Hk=32, D=128, B=32, rot=128, interleaved=False, stretch=4.0,
             dtype="bf16"),
        # the small model's decode step, fp32 result
        dict(name="decode_q8_tiny", op="decode_q8", S=4, H=8, Hk=8, D=64, B=16, lo=1, hi=200,
             dtype="fp16", out="fp32"),
        # a serving batch of grouped-query heads, contexts of mixed lengths
        dict(name="decode_q8_gqa", op="decode_q8", S=128, H=32, Hk=8, D=128, B=16, lo=16, hi=8192,
             dtype="bf16", out="bf16"),
        # long contexts, one kv head per query head, larger pages
        dict(name="decode_q8_long_mha", op="decode_q8", S=16, H=32, Hk=32, D=128, B=32, lo=8192,
             hi=32768, dtype="bf16", out="bf16"),
        # drafted tokens to verify on a small grouped-query model
        dict(name="chunk_q8_verify", op="chunk_q8", S=16, q_lo=1, q_hi=8, H=16, Hk=4, D=64, B=16,
             lo=8, hi=1000, dtype="fp16", out="fp16"),
        # a chunk of each prompt of a serving batch, behind what is cached
        dict(name="chunk_q8_gqa", op="chunk_q8", S=8, q_lo=100, q_hi=512, H=32, Hk=8, D=128, B=16,
             lo=1000, hi=8192, dtype="bf16", out="bf16"),
        # large chunks of long documents, one kv head per query head
        dict(name="chunk_q8_long_mha", op="chunk_q8", S=2, q_lo=2048, q_hi=2048, H=32, Hk=32,
             D=128, B=32, lo=12000, hi=16384, dtype="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "decode_q8", "chunk_q8"])
    Hk = rng.choice([1, 2, 4, 8, 16, 32])
    G = rng.choice([g for g in (1, 2, 4, 8) if g * Hk <= 64])
    D = rng.choice([64, 128])
    B = rng.choice([16, 32])
    dt = rng.choice(["bf16", "fp16"])
    case = dict(op=op, H=G * Hk, Hk=Hk, D=D, B=B, dtype=dt)
    if op in ("append", "append_q8"):
        most = max(1, min(16384, 8 * 10 ** 7 // ((G + 2) * Hk * D)))    # new tokens
        hi = rng.choice([1, _log(rng, 1, min(2048, most))])
        S = _log(rng, 1, min(512, most // hi))
        rot = rng.choice([D, D, D // 2, D // 4])
        return dict(case, S=S, lo=_log(rng, 1, hi), hi=hi, before=_log(rng, 1, 16384),
                    pad=rng.choice([0, 0, rng.randint(1, 9)]), rot=rot,
                    interleaved=rng.random() < 0.5, stretch=rng.choice([1.0, 1.0, 2.0, 8.0]))
    if op == "decode_q8":
        hi = _log(rng, 1, 32768)
        S = _log(rng, 1, max(1, min(256, 10 ** 9 // (Hk * D * hi))))
        return dict(case, S=S, lo=_log(rng, 1, hi), hi=hi, out=rng.choice([dt, dt, "fp32"]))
    q_hi = _log(rng, 1, 2048)
    hi = max(q_hi, _log(rng, 1, 16384))
    S = _log(rng, 1, max(1, min(64, 10 ** 9 // (G * Hk * q_hi * hi),
                                5 * 10 ** 8 // (G * Hk * D * hi))))
    return dict(case, S=S, q_lo=_log(rng, 1, q_hi), q_hi=q_hi, lo=_log(rng, 1, hi), hi=hi, out=dt)


def _spread(tag, case, lo, hi):
    """A number per sequence, from the case alone; the largest is `hi`."""
    r = random.Random("%s %s %d %d %d" % (tag, case["op"], case["S"], lo, hi))
    n = [r.randint(lo, hi) for _ in range(case["S"])]
    n[r.randrange(case["S"])] = hi
    return n


def _appended(case):
    """Of every sequence: tokens cached before, and new ones."""
    return _spread("before", case, 0, case["before"]), _spread("new", case, case["lo"], case["hi"])


def _contexts(case):
    """Of every sequence: its new tokens (the last ones) and its context."""
    q = _spread("chunk", case, case["q_lo"], case["q_hi"])
    return q, [max(a, b) for a, b in zip(q, _spread("context", case, case["lo"], case["hi"]))]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _rope_table(positions, rot, stretch):
    """fp32 [positions, rot]: cosines, then sines, of angles formed in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] / stretch * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _quantised(gen, blocks, case, channels):
    """8-bit pages as an earlier calibration left them (scales of any size),
    from values whose channels differ in size."""
    x = torch.randn((blocks, case["B"], case["Hk"], case["D"]), generator=gen, device="cuda")
    if channels:
        x *= torch.randn((case["Hk"], case["D"]), generator=gen, device="cuda").mul_(0.5).exp_()
    scale = (x.abs().amax((1, 3)) / _E4M3_MAX).clamp_(min=_LEAST_SCALE)
    x = x.div_(scale[:, None, :, None]).clamp_(-_E4M3_MAX, _E4M3_MAX)
    return x.to(_E4M3), scale


def _prepare_append(case, gen):
    before, new = _appended(case)
    S, H, Hk, D, B = (case[k] for k in ("S", "H", "Hk", "D", "B"))
    dt = _TYPES[case["dtype"]]
    first = [b % B for b in before]                    # rows held by the first page
    pages = [(f + n + B - 1) // B for f, n in zip(first, new)]
    spare = sum(pages) // 4 + 1                        # other requests' pages
    blocks = sum(pages) + spare
    perm = torch.randperm(blocks, generator=gen, device="cuda")
    slots, positions, at = [], [], 0
    for b, f, n, c in zip(before, first, new, pages):
        slots += [at * B + f + i for i in range(n)]
        positions += list(range(b, b + n))
        at += c
    slots = _ints(slots, torch.int64)
    slots = torch.cat([perm[slots // B] * B + slots % B,
                       _ints([-1] * case["pad"], torch.int64)])
    T = slots.shape[0]
    qkv = torch.randn((T, H + 2 * Hk, D), generator=gen, device="cuda")
    qkv[:, H:H + Hk] *= torch.randn((Hk, D), generator=gen, device="cuda").mul_(0.5).exp_()
    qkv = qkv.to(dt)                                   # the fused projection's output
    st = dict(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], slots=slots,
              positions=_ints(positions + [0] * case["pad"]),
              rope=_rope_table(case["before"] + case["hi"], case["rot"], case["stretch"]),
              interleaved=case["interleaved"], q_out=torch.zeros((T, H, D), device="cuda", dtype=dt))
    if case["op"] == "append":
        st["k_pool"], st["v_pool"] = (torch.randn((blocks, B, Hk, D), generator=gen, device="cuda",
                                                  dtype=dt) for _ in range(2))
        return st
    for name in ("k", "v"):
        # pages that this append filled so far: a power of two per block and
        # head, fitted to fewer and so mostly smaller values than now
        x = torch.randn((blocks, B, Hk, D), generator=gen, device="cuda")
        x *= torch.rand((blocks, 1, Hk, 1), generator=gen, device="cuda").mul_(2).sub_(2).exp2_()
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 3)) / _E4M3_MAX)))
        st[name + "_pool"] = (x / scale[:, None, :, None]).clamp_(-_E4M3_MAX, _E4M3_MAX).to(_E4M3)
        st[name + "_scale"] = scale
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] in ("append", "append_q8"):
        return dict(_prepare_append(case, gen), op=case["op"], case=dict(case))
    dt, B, S, H, D = _TYPES[case["dtype"]], case["B"], case["S"], case["H"], case["D"]
    if case["op"] == "decode_q8":
        n_q, lens = None, _spread("context", case, case["lo"], case["hi"])
        rows = S
    else:
        n_q, lens = _contexts(case)
        rows = sum(n_q)
    pages = [(n + B - 1) // B for n in lens]
    width = max(pages)
    perm = torch.randperm(sum(pages), generator=gen, device="cuda").to(torch.int32)
    tables = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    tables[torch.arange(width, device="cuda")[None, :] < _ints(pages)[:, None]] = perm
    k_pool, k_scale = _quantised(gen, sum(pages), case, True)
    v_pool, v_scale = _quantised(gen, sum(pages), case, False)
    st = dict(op=case["op"], case=dict(case), k_pool=k_pool, v_pool=v_pool, k_scale=k_scale,
              v_scale=v_scale, tables=tables, lens=_ints(lens), max_len=max(lens),
              scale=1.0 / math.sqrt(D),
              q=torch.randn((rows, H, D), generator=gen, device="cuda", dtype=dt),
              out=torch.zeros((rows, H, D), device="cuda", dtype=_TYPES[case["out"]]))
    if n_q is not None:
        starts = [0]
        for n in n_q:
            starts.append(starts[-1] + n)
        st.update(q_start=_ints(starts), max_q=max(n_q))
    return st


# ------------------------------------------------------------ plain forms

def _rotated(x, st):
    """fp32 x with the leading `rot` elements of every head rotated in pairs."""
    x = x.float()
    rot = st["rope"].shape[1]
    c, s = st["rope"][st["positions"].long()][:, None].chunk(2, 2)
    h = x[..., :rot]
    a, b = (h[..., 0::2], h[..., 1::2]) if st["interleaved"] else h.chunk(2, -1)
    pair = (a * c - b * s, a * s + b * c)
    h = torch.stack(pair, -1).flatten(-2) if st["interleaved"] else torch.cat(pair, -1)
    return torch.cat([h, x[..., rot:]], -1)


def _append_q8_plain(x, slots, pool, scale):
    """Rows x (fp32 [T, Hk, D]) into 8-bit pages.  A block's rows ahead of the
    first one written are kept; its scale is the least power of two that holds
    the new rows, or the old one where rows are kept and it is larger."""
    nb, B, Hk, D = pool.shape
    live = slots >= 0
    # what is skipped goes to a block of its own, behind the others
    block = torch.where(live, slots // B, nb)
    first = torch.full((nb + 1,), B, device=x.device).scatter_reduce(0, block, slots % B, "amin")
    most = torch.zeros((nb + 1, Hk), device=x.device)
    most = most.scatter_reduce(0, block[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")[:nb]
    first = first[:nb, None]
    m, e = torch.frexp(most)
    new = torch.exp2((e - 9 + (m > _E4M3_MAX / 512).int()).float())
    new = torch.where(most > 0, new, 0.0).clamp(min=_LEAST_SCALE)
    new = torch.where(first == B, scale, torch.where(first > 0, torch.maximum(scale, new), new))
    row = torch.arange(B, device=x.device)[None, :, None, None]
    kept = (pool.float() * (scale / new)[:, None, :, None]).to(_E4M3).view(torch.uint8)
    kept = torch.where(row < first[:, :, None, None], kept, pool.view(torch.uint8))
    codes = x / torch.cat([new, new.new_ones(1, Hk)])[block][..., None]
    codes = codes.clamp(-_E4M3_MAX, _E4M3_MAX).to(_E4M3).view(torch.uint8)
    kept = torch.cat([kept, kept.new_zeros(1, B, Hk, D)]).view(-1, Hk, D)
    kept[torch.where(live, slots, nb * B)] = codes
    pool.view(torch.uint8).copy_(kept[:nb * B].view(nb, B, Hk, D))
    scale.copy_(new)


def _plain_append(st):
    live = st["slots"] >= 0
    st["q_out"].copy_(torch.where(live[:, None, None], _rotated(st["q"], st).to(st["q_out"].dtype),
                                  st["q_out"]))
    k, v = _rotated(st["k"], st), st["v"].float()
    if st["op"] == "append_q8":
        _append_q8_plain(k, st["slots"], st["k_pool"], st["k_scale"])
        _append_q8_plain(v, st["slots"], st["v_pool"], st["v_scale"])
        return
    for x, pool in ((k, st["k_pool"]), (v, st["v_pool"])):
        rows = pool.view(-1, *pool.shape[2:])
        at = st["slots"].clamp(min=0)
        # what is skipped writes the first row's own value or its new one
        last = torch.where(live, at, -1)
        hit = (last == 0).any()
        zero = torch.where(hit, x[(last == 0).int().argmax()].to(rows.dtype), rows[0])
        rows[at] = torch.where(live[:, None, None], x.to(rows.dtype), zero)


def _values(st, name, L):
    """fp32 [S, Hk, L, D]: the values that the 8-bit pages stand for."""
    pool, scale, B = st[name + "_pool"], st[name + "_scale"], st["case"]["B"]
    t = torch.arange(L, device=pool.device)
    block = st["tables"].long().clamp(min=0)[:, t // B]               # [S, L]
    rows = pool.view(torch.uint8).view(-1, *pool.shape[2:])[block * B + t % B]
    return (rows.view(_E4M3).float() * scale[block][..., None]).transpose(1, 2)


def _plain_attention(st):
    q, L, lens = st["q"].float(), st["max_len"], st["lens"].long()
    T, H, D = q.shape
    S = lens.shape[0]
    if st["op"] == "decode_q8":
        Q, at = 1, torch.arange(S, device=q.device)[:, None]
        n_q = torch.ones_like(lens)
    else:
        Q, starts = st["max_q"], st["q_start"].long()
        n_q = starts[1:] - starts[:-1]
        at = (starts[:-1, None] + torch.arange(Q, device=q.device)).clamp(max=T - 1)
    Hk = st["k_pool"].shape[2]
    # rows of a kv head: its query heads' tokens [S, Hk, G * Q, D]
    x = q[at].view(S, Q, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, -1, D)
    x = torch.matmul(x, _values(st, "k", L).transpose(2, 3)).mul_(st["scale"])
    x = x.view(S, Hk, H // Hk, Q, L)
    last = lens[:, None] - n_q[:, None] + torch.arange(Q, device=q.device)
    hidden = torch.arange(L, device=q.device) > last[..., None]       # [S, Q, L]
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    o = torch.matmul(x.view(S, Hk, -1, L), _values(st, "v", L))
    o = o.view(S, Hk, H // Hk, Q, D).permute(0, 3, 1, 2, 4).reshape(S, Q, H, D)
    if st["op"] == "decode_q8":
        st["out"].copy_(o[:, 0])
    else:
        t = torch.arange(T, device=q.device)
        s = torch.searchsorted(starts[1:].contiguous(), t, right=True)
        st["out"].copy_(o[s, t - starts[s]])


def run(st):
    if own:
        import paged_kv_decode_26_gb300 as pkv
    op = st["op"]
    if op == "append":
        if own:
            pkv.kv_append_rope(st["k_pool"], st["v_pool"], st["k"], st["v"], st["slots"],
                               st["positions"], st["rope"], st["q"], st["q_out"],
                               interleaved=st["interleaved"])
        else:
            _plain_append(st)
        return {k: st[k] for k in ("k_pool", "v_pool", "q_out")}
    if op == "append_q8":
        if own:
            pkv.kv_append_rope_q8(st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"],
                                  st["k"], st["v"], st["slots"], st["positions"], st["rope"],
                                  st["q"], st["q_out"], interleaved=st["interleaved"])
        else:
            _plain_append(st)
        return {k: st[k] for k in ("k_pool", "v_pool", "k_scale", "v_scale", "q_out")}
    if op == "decode_q8":
        if own:
            pkv.paged_attn_decode_q8(st["out"], st["q"], st["k_pool"], st["v_pool"],
                                     st["k_scale"], st["v_scale"], st["tables"], st["lens"],
                                     st["scale"], st["max_len"])
        else:
            _plain_attention(st)
        return st["out"]
    if own:
        pkv.paged_attn_multi_query_q8(st["out"], st["q"], st["q_start"], st["k_pool"],
                                      st["v_pool"], st["k_scale"], st["v_scale"], st["tables"],
                                      st["lens"], st["scale"], st["max_q"], st["max_len"])
    else:
        _plain_attention(st)
    return st["out"]


# ----------------------------------------------------------- 64-bit values

def _turn64(x, st, t):
    """Token t's heads, in 64 bits, as complex numbers times e^(i angle)."""
    rot = st["rope"].shape[1]
    turn = torch.complex(*st["rope"][st["positions"][t].long()].double().view(-1, 2, rot // 2)
                         .unbind(1))[:, None]
    x = x[t].double()
    if st["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _round_e4m3(x):
    """The nearest number of 4 exponent and 3 mantissa bits, ties to even."""
    least = torch.full_like(x, -6.0)
    step = torch.exp2(torch.maximum(torch.floor(torch.log2(x.abs().clamp(min=1e-300))), least) - 3)
    return (torch.round(x / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)


def _exact_append(st, case):
    B = case["B"]
    slots = st["slots"]
    live = torch.nonzero(slots >= 0)[:, 0]
    st["q_out"] = st["q_out"].double()
    st["q_out"][live] = _turn64(st["q"], st, live)
    out = {}
    for name, x in (("k", _turn64(st["k"], st, live)), ("v", st["v"][live].double())):
        pool = st[name + "_pool"].double()
        at = slots[live]
        if case["op"] == "append":
            pool.view(-1, *pool.shape[2:])[at] = x
            out[name + "_pool"] = pool
            continue
        scale = st[name + "_scale"].double()
        blocks, of = torch.unique(at // B, return_inverse=True)
        # the block's rows that this call writes, NaN elsewhere
        rows = torch.full((blocks.shape[0], *pool.shape[1:]), math.nan, dtype=torch.float64,
                          device="cuda")
        rows[of, at % B] = x
        written = ~rows[:, :, 0, 0].isnan()
        first = written.int().argmax(1)
        peak = rows.nan_to_num(nan=0.0).abs().amax((1, 3))
        # (by comparison: a logarithm may fall to either side of a whole number)
        need = torch.exp2(torch.floor(torch.log2(peak.clamp(min=1e-300) / _E4M3_MAX)) - 1)
        for _ in range(3):
            need = torch.where(need * _E4M3_MAX < peak, 2 * need, need)
        need = need.clamp(min=_LEAST_SCALE)
        old = scale[blocks]
        new = torch.where((first > 0)[:, None], torch.maximum(old, need), need)
        keep = torch.arange(B, device="cuda")[None, :] < first[:, None]
        was = pool[blocks]
        held = _round_e4m3(was * (old / new)[:, None, :, None])
        page = torch.where(keep[..., None, None], held, was)
        page = torch.where(written[..., None, None], _round_e4m3(rows / new[:, None, :, None]), page)
        pool[blocks] = page
        scale[blocks] = new
        out[name + "_pool"], out[name + "_scale"] = pool, scale
    return dict(out, q_out=st["q_out"])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("append", "append_q8"):
        return _exact_append(st, case)
    B, Hk, D, S = case["B"], case["Hk"], case["D"], case["S"]
    G = case["H"] // Hk
    if case["op"] == "decode_q8":
        starts = list(range(S + 1))
    else:
        starts = st["q_start"].tolist()
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    for s in range(S):
        n, a, b = int(st["lens"][s]), starts[s], starts[s + 1]
        pages = st["tables"][s, :(n + B - 1) // B].long()
        hidden = torch.ones(b - a, n, dtype=torch.bool, device="cuda").triu(n - (b - a) + 1)
        for h in range(Hk):
            k, v = ((st[x + "_pool"][:, :, h].view(torch.uint8)[pages].view(_E4M3).double()
                     * st[x + "_scale"][pages, h].double()[:, None, None]).view(-1, D)[:n]
                    for x in ("k", "v"))
            for g in range(G):
                x = st["q"][a:b, h * G + g].double() @ k.T * st["scale"]
                x = x.masked_fill(hidden, -math.inf)
                p = torch.exp(x - x.max(-1, keepdim=True).values)
                out[a:b, h * G + g] = (p @ v) / p.sum(-1, keepdim=True)
    return out


# ------------------------------------------------------------ what it costs

def work(case):
    """Each input that the operator needs read once, each output written once.
    8-bit blocks: the scales of those touched, and no rows that are kept."""
    H, Hk, D, B, S = (case[k] for k in ("H", "Hk", "D", "B", "S"))
    e = 2
    if case["op"] in ("append", "append_q8"):
        before, new = _appended(case)
        T = sum(new)
        pages = sum((b % B + n + B - 1) // B for b, n in zip(before, new))
        held = e if case["op"] == "append" else 1
        scales = 0 if case["op"] == "append" else 2 * 2 * 4 * Hk * pages
        return {"bytes": T * D * (2 * H * e + 2 * Hk * (e + held)) + scales
                + T * (8 + 4 + 4 * case["rot"]), "flops": 3 * T * (H + Hk) * case["rot"]}
    eo = 4 if case["out"] == "fp32" else 2
    if case["op"] == "decode_q8":
        lens = _spread("context", case, case["lo"], case["hi"])
        rows, seen = S, sum(lens)
    else:
        n_q, lens = _contexts(case)
        rows, seen = sum(n_q), sum(q * n - q * (q - 1) // 2 for q, n in zip(n_q, lens))
    pages = sum((n + B - 1) // B for n in lens)
    return {"bytes": 2 * sum(lens) * Hk * D + pages * (4 + 2 * 4 * Hk) + rows * H * D * (e + eo)
            + 8 * S, "flops": 4 * H * D * seen}

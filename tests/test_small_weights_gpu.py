"""Many keys of small weight beside one of large weight (attention sinks): the
small ones' sum has to arrive whole in every operator, fp16 caches included,
whose smallest numbers are far above those of fp32 and bf16.

Channel d of V is 1 at the keys of class d % 8 and 0 elsewhere, the large key's
row is 0, so an output element is the sum of one class's weights: A is that
sum itself, and out_bound (tests/cache_ref.py) asks for it to the rounding of
a weight.  Where weights leave the softmax as fp16, they are carried relative
to 2^-11 of the largest one, so the spacing of fp16's smallest numbers, 2^-24,
is 2^-35 of the largest weight and costs a key at most half of that: n 2^-36
per class of n keys, added to the bound.  Outputs of the first rows are below
2^-14, where fp16 outputs themselves are spaced by 2^-24 whatever their value:
a rounding of at most 2^-25 there, added for fp16 outputs."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
KINDS = [(FP, FP), (FP, F32), (BF, BF), (BF, F32)]


def _sink(n, H, Hk, D, dtype):
    """q [H, D], k, v [n, Hk, D]: key 0's weight is the largest; class c's are
    2^-(10 + 1.3 c) of it, (c a key's index mod 8)."""
    q = torch.zeros(H, D)
    q[:, 0] = 16.0
    q[:, 1] = 1.0
    c = torch.arange(n) % 8
    x = -(10 + 1.3 * c.double()) * math.log(2.0)        # natural units, scale 1
    k = torch.zeros(n, Hk, D)
    hi = (x / 16).float().to(dtype).double()
    k[:, :, 0] = hi.float()[:, None]
    k[:, :, 1] = (x - 16 * hi).float()[:, None]
    k[0] = 0
    v = torch.zeros(n, Hk, D)
    for d in range(D):
        v[c == d % 8, :, d] = 1.0
    v[0] = 0
    return q.to(dtype), k.to(dtype), v.to(dtype)


def _check(out, o, bound, dtype, n, what):
    floor = (n / 8 + 1) * 2.0 ** -36 if dtype == FP else 0.0
    ref.check(out, o, bound + floor + (2.0 ** -25 if out.dtype == FP else 0.0), what)


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_keeps_small_weights(D, dtype, out_dtype):
    n, H, Hk = 1500, 2, 1
    q, k, v = _sink(n, H, Hk, D, dtype)
    q = q.expand(n, H, D).contiguous()
    out = torch.empty(n, H, D, dtype=out_dtype, device="cuda")
    pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(),
                    torch.tensor([0, n], dtype=torch.int32, device="cuda"), 1.0, n)
    hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
    for h in range(H):
        o, _, A, d = ref.attend(q[:, h], k[:, 0], v[:, 0], 1.0, hidden)
        _check(out[:, h], o, ref.out_bound(o, A, d, dtype, out_dtype, once=out_dtype != F32),
               dtype, n, f"head {h}")


def _paged(n, H, Hk, D, dtype, members, prefix):
    """Sequences of n tokens whose first `prefix` lie in the same pages."""
    B = 16
    q, k, v = _sink(n, H, Hk, D, dtype)
    pages, common = (n + B - 1) // B, prefix // B
    blocks = common + members * (pages - common)
    tables = torch.full((members, pages), -1, dtype=torch.int32)
    kp = torch.full((blocks, B, Hk, D), float("nan"), dtype=dtype)
    vp = kp.clone()
    for s in range(members):
        for j in range(pages):
            b = j if j < common else common + s * (pages - common) + j - common
            rows = min(B, n - j * B)
            kp[b, :rows], vp[b, :rows] = k[j * B:j * B + rows], v[j * B:j * B + rows]
            tables[s, j] = b
    return (q.expand(members, H, D).contiguous(), k, v, kp.cuda(), vp.cuda(), tables.cuda(),
            torch.full((members,), n, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_weights_decode_keeps_small_weights(D, dtype, out_dtype):
    n, H, Hk = 6000, 2, 2
    q, k, v, kp, vp, tables, lens = _paged(n, H, Hk, D, dtype, 1, 0)
    out = torch.empty(1, H, D, dtype=out_dtype, device="cuda")
    w = torch.zeros(1, n, device="cuda")
    pkv.paged_attn_decode_weights(out, q.cuda(), kp, vp, tables, lens, w, 1.0, n)
    o, bound, ws = ref.decode(q, [k], [v], 1.0, out_dtype)
    _check(out, o, bound, dtype, n, "out")
    ref.check(w[0], ws[0][0], ws[0][1] + 2.0 ** -23 * ws[0][0], "weights")


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
def test_weights_decode_keeps_small_weights_in_long_runs(dtype, out_dtype):
    """Enough sequences (of the same pages) that each is one piece."""
    n, H, Hk, D, S = 1500, 2, 2, 64, 900
    q, k, v, kp, vp, tables, lens = _paged(n, H, Hk, D, dtype, 1, 0)
    out = torch.empty(S, H, D, dtype=out_dtype, device="cuda")
    w = torch.zeros(S, n, device="cuda")
    pkv.paged_attn_decode_weights(out, q.cuda().expand(S, H, D).contiguous(), kp, vp,
                                  tables.expand(S, -1).contiguous(), lens.expand(S).contiguous(),
                                  w, 1.0, n)
    o, bound, ws = ref.decode(q, [k], [v], 1.0, out_dtype)
    _check(out, o.expand(S, H, D), bound, dtype, n, "out")
    ref.check(w, ws[0][0].expand(S, n), ws[0][1] + 2.0 ** -23 * ws[0][0], "weights")


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_shared_decode_keeps_small_weights(D, dtype, out_dtype):
    n, H, Hk = 3000, 4, 2
    q, k, v, kp, vp, tables, lens = _paged(n, H, Hk, D, dtype, 3, 2000)
    out = torch.empty(3, H, D, dtype=out_dtype, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pkv.paged_attn_decode_shared(out, q.cuda(), kp, vp, tables, lens, ints([0, 3]), ints([2000]),
                                 1.0, n, 3, 2000)
    o, bound, _ = ref.decode(q, [k] * 3, [v] * 3, 1.0, out_dtype, once=out_dtype != F32)
    _check(out, o, bound, dtype, n, "out")

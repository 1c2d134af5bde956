"""Values of V near the end of bf16's range, where the running reference of the
softmax is below the largest score: a weight above 1 on its way into the second
product would leave fp32's range although the result, a mean of the values, is
finite.  Three keys carry the weight, the later ones above the first by less
than makes a kernel move its reference; against the 64-bit form with the
tolerances of tests/cache_ref.py.  Scores of 2^21 (the second base) are resolved
to 1/4 only, which those tolerances allow for: there the result has to be
finite and within them."""
import math

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref
from tests.test_large_scores_gpu import _pages

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
N, HEAVY = 700, {0: 0.0, 200: 4.0, 330: 7.0}       # key: score above the first, log2 units


def _rows(rows, H, Hk, D, base):
    """q [rows, H, D], k, v [N, Hk, D], scale 1 in log2 units."""
    q = torch.zeros(rows, H, D)
    q[..., 0], q[..., 1] = 2.0 ** 10, 1.0
    k = torch.zeros(N, Hk, D)
    k[..., 0] = base / 2.0 ** 10
    k[..., 1] = -64.0
    for t, x in HEAVY.items():
        k[t, :, 1] = x
    g = torch.Generator().manual_seed(D)
    v = torch.sign(torch.randn(N, Hk, D, generator=g)) * (1 + torch.rand(N, Hk, D, generator=g))
    return q.to(BF), k.to(BF), (v * 2.0 ** 124).to(BF), math.log(2.0)


KINDS = [(D, o, b) for D in (64, 128) for o in (BF, F32) for b in (0.0, 2.0 ** 21)]


@pytest.mark.parametrize("D,out_dtype,base", KINDS)
def test_prompt(D, out_dtype, base):
    H, Hk = 4, 2
    q, k, v, scale = _rows(N, H, Hk, D, base)
    out = torch.empty(N, H, D, dtype=out_dtype, device="cuda")
    pkv.attn_prompt(out, q.cuda(), k.cuda(), v.cuda(),
                    torch.tensor([0, N], dtype=torch.int32, device="cuda"), scale, N)
    hidden = torch.ones(N, N, dtype=torch.bool).triu(1)
    for h in range(H):
        o, _, A, d = ref.attend(q[:, h], k[:, h // 2], v[:, h // 2], scale, hidden)
        ref.check(out[:, h], o, ref.out_bound(o, A, d, BF, out_dtype, out_dtype != F32))


@pytest.mark.parametrize("D,out_dtype,base", KINDS)
@pytest.mark.parametrize("S", [3, 600])
def test_weights_decode(D, out_dtype, base, S):
    lens, H, Hk = [N, 250, 335] * (S // 3), 4, 2
    q, k, v, scale = _rows(S, H, Hk, D, base)
    kp, vp, tables, ln = _pages(lens, 16, k, v)
    out = torch.empty(S, H, D, dtype=out_dtype, device="cuda")
    pkv.paged_attn_decode_weights(out, q.cuda(), kp, vp, tables, ln, torch.zeros(S, N).cuda(),
                                  scale, N)
    o, bound, _ = ref.decode(q[:3], [k[:n] for n in lens[:3]], [v[:n] for n in lens[:3]], scale,
                             out_dtype)
    ref.check(out, o.repeat(S // 3, 1, 1), bound.repeat(S // 3, 1, 1))


@pytest.mark.parametrize("D,out_dtype,base", KINDS)
@pytest.mark.parametrize("once", [0, 1])
def test_shared_decode(D, out_dtype, base, once):
    lens, H, Hk, prefix = [N, 530, 640], 4, 2, 512
    q, k, v, scale = _rows(3, H, Hk, D, base)
    kp, vp, tables, ln = _pages(lens, 16, k, v)
    out = torch.empty(3, H, D, dtype=out_dtype, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pkv.set_tuning(shared_prefix=once)
    try:
        pkv.paged_attn_decode_shared(out, q.cuda(), kp, vp, tables, ln, ints([0, 3]),
                                     ints([prefix]), scale, N, 3, prefix)
    finally:
        pkv.reset_tuning()
    o, bound, _ = ref.decode(q, [k[:n] for n in lens], [v[:n] for n in lens], scale, out_dtype,
                             once=out_dtype != F32)
    ref.check(out, o, bound)

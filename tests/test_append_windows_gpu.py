"""8-bit appends at numbers of tokens and heads around those from which a CTA takes windows
of several tokens, runs that straddle them among them, against the plain form."""
import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import q8_ref as ref

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


@pytest.mark.parametrize("D,B,H,Hk,around", [
    # tokens x CTAs a token against six CTAs on each of 152 SMs
    (64, 16, 4, 1, 456), (64, 16, 0, 1, 912), (64, 32, 8, 2, 304), (128, 16, 32, 8, 101),
    (128, 16, 16, 16, 53), (128, 32, 32, 32, 14), (128, 32, 0, 32, 14)])
@pytest.mark.parametrize("decode", [False, True])
def test_numbers_of_tokens(D, B, H, Hk, around, decode):
    for n in (around - 2, around - 1, around, around + 1, 2 * around + 3):
        torch.cuda.synchronize()
        pkv.device_errors(clear=True)
        gen = torch.Generator().manual_seed(81 + n)
        if decode:                                 # a token each
            blocks = n + 2
            slots = (torch.randperm(blocks, generator=gen)[:n] * B +
                     torch.randint(0, B, (n,), generator=gen)).tolist()
        else:                                      # two prompts
            first, second = n // 3, n - n // 3
            blocks = (5 + first) // B + (11 + second) // B + 3
            at = ((5 + first) // B + 1) * B + 11
            slots = list(range(5, 5 + first)) + list(range(at, at + second))
        q, k, v = (torch.randn(n, h, D, generator=gen) for h in (max(H, 1), Hk, Hk))
        v *= (torch.rand(n, 1, 1, generator=gen) * 4).exp2()
        q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
        pool = ref.round_e4m3(torch.randn(blocks, B, Hk, D, generator=gen).double() * 60)
        scale = torch.randint(-9, -5, (blocks, Hk), generator=gen).float().exp2()
        kp, vp = pool.to(E4).cuda(), pool.to(E4).cuda()
        ks, vs = scale.clone().cuda(), scale.clone().cuda()
        pos = torch.arange(n, dtype=torch.int32)
        table = ref.table64(n, D)
        q_out = torch.full_like(q, 7.0, device="cuda")
        pkv.kv_append_rope_q8(kp, vp, ks, vs, k.cuda(), v.cuda(), torch.tensor(slots).cuda(), pos.cuda(),
                              table.cuda(), q.cuda() if H else None, q_out if H else None)
        torch.cuda.synchronize()
        assert pkv.device_errors(clear=True) == 0
        zero = torch.zeros(n, Hk, D, dtype=torch.float64)
        w = ref.append_q8(pool, scale.double(), v.double(), zero, slots)
        assert torch.equal(vp.cpu().double(), w[0]) and torch.equal(vs.cpu().double(), w[1]), n
        kr, err = ref.rotate(k, table, pos, False)
        # a step of the values, or of numbers below 2^-6 of the scale
        s = torch.tensor(slots)
        got = (kp.cpu().double() * ks.cpu().double()[:, None, :, None]).view(-1, Hk, D)[s]
        step = torch.maximum(kr.abs() * 2.0 ** -4, ks.cpu().double()[s // B][..., None] * 2.0 ** -10)
        assert ((got - kr).abs() <= step * (1 + 2.0 ** -20) + err).all(), n
        if H:
            qr, err = ref.rotate(q, table, pos, False)
            assert ((q_out.cpu().double() - qr).abs() <= err + 2.0 ** -8 * (qr.abs() + err)).all(), n

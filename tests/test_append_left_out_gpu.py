"""8-bit appends with tokens that are left out (a negative slot, one beyond the pool, a
position outside the table) anywhere in the call: the same pages, scales and outputs as
without those tokens."""
import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from paged_kv_decode_26_gb300 import _lib
from tests import q8_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
E4 = torch.float8_e4m3fn
ROWS = 5000                                       # of the rotation table


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


def _layout(gen, seqs, B, gaps, kinds):
    """(slots, positions, alive) of sequences of (rows held, new tokens), with runs of
    left-out tokens of the lengths `gaps` strewn between, the blocks they take, and the
    flags that they raise."""
    def pick(n):
        return int(torch.randint(0, n, (1,), generator=gen))

    slots, pos, alive, blocks, flags = [], [], [], 0, 0
    for held, n in seqs:
        first = blocks * B + held % B
        blocks += (held % B + n + B - 1) // B
        for i in range(n):
            if i == 1 or pick(9) == 0:
                for _ in range(gaps[pick(len(gaps))]):
                    kind = kinds[pick(len(kinds))]
                    slots.append(-1 if kind == "pad" else (1 << 33) if kind == "beyond" else first + i)
                    pos.append(ROWS + pick(9) if kind == "position" else 0)
                    alive.append(False)
                    flags |= {"pad": 0, "beyond": _lib.DEVERR_SLOT, "position": _lib.DEVERR_POSITION}[kind]
            slots.append(first + i)
            pos.append((held + i) % ROWS)
            alive.append(True)
    return slots, pos, alive, blocks, flags


@pytest.mark.parametrize("kinds", [("pad",), ("beyond",), ("position",), ("pad", "beyond", "position")])
@pytest.mark.parametrize("seqs,gaps", [
    ([(5, 9), (0, 3)], [1]),
    ([(3, 30), (16, 40), (31, 1), (0, 17)], [1, 2, 5]),
    ([(7, 20), (0, 33)], [20, 40, 300, 700]),
    ([(i, 1 + i % 5) for i in range(90)], [1, 3, 17]),
    ([(11, 500), (0, 700), (40, 90)], [1, 2, 15, 16, 31, 32, 33, 400]),
])
@pytest.mark.parametrize("D,B,Hk", [(64, 16, 2), (128, 32, 1), (128, 16, 8)])
def test_left_out_tokens_change_nothing(D, B, Hk, seqs, gaps, kinds):
    _clean()
    gen = torch.Generator().manual_seed(41)
    H = 2 * Hk
    slots, pos, alive, blocks, flags = _layout(gen, seqs, B, gaps, kinds)
    T = len(slots)
    keep = torch.tensor(alive).nonzero()[:, 0]
    assert 0 < len(keep) < T
    qkv = torch.randn(T, H + 2 * Hk, D, generator=gen)
    qkv *= (torch.rand(T, 1, 1, generator=gen) * 4).exp2()          # scales grow and stay
    qkv = qkv.to(BF)
    # what is left out is far larger than the others
    qkv[~torch.tensor(alive)] *= 64.0
    table = ref.table64(ROWS, D, dev="cuda")
    pool = ref.round_e4m3(torch.randn(blocks, B, Hk, D, generator=gen).double() * 60).to(E4)
    scale = torch.randint(-9, -4, (blocks, Hk), generator=gen).float().exp2()
    slots, pos = torch.tensor(slots), torch.tensor(pos, dtype=torch.int32)

    def call(at):
        x = qkv[at].cuda()
        st = dict(kp=pool.clone().cuda(), vp=pool.clone().cuda(), ks=scale.clone().cuda(),
                  vs=scale.clone().cuda(), q=torch.full((len(at), H, D), 7.0, dtype=BF, device="cuda"),
                  k=torch.full((len(at), Hk, D), 7.0, dtype=BF, device="cuda"))
        pkv.kv_append_rope_q8(st["kp"], st["vp"], st["ks"], st["vs"], x[:, H:H + Hk], x[:, H + Hk:],
                              slots[at].cuda(), pos[at].cuda(), table, x[:, :H], st["q"], st["k"])
        return st

    want = call(keep)
    assert _clean() == 0
    # (the form knows no rotation: the values')
    zero = torch.zeros(len(keep), Hk, D, dtype=torch.float64)
    w = ref.append_q8(pool.double(), scale.double(), qkv[keep, H + Hk:].double(), zero,
                      slots[keep].tolist())
    assert torch.equal(want["vs"].cpu().double(), w[1])
    assert torch.equal(want["vp"].cpu().double(), w[0])
    got = call(torch.arange(T))
    assert _clean() == flags
    for name in ("kp", "vp", "ks", "vs"):
        assert torch.equal(got[name].view(torch.uint8), want[name].view(torch.uint8)), name
    for name in ("q", "k"):
        assert torch.equal(got[name][keep.cuda()], want[name]), name
        rest = (~torch.tensor(alive)).nonzero()[:, 0].cuda()
        assert (got[name][rest] == 7.0).all(), name


@pytest.mark.parametrize("n", [3, 400])
def test_blocks_of_left_out_tokens_alone_keep_their_scales(n):
    """Tokens outside the table, to a block's first row and on: nothing is written."""
    _clean()
    Hk, D, B = 2, 64, 16
    blocks = n // B + 1
    gen = torch.Generator().manual_seed(42)
    k, v = (torch.randn(n, Hk, D, generator=gen).to(BF).cuda() for _ in range(2))
    kp, vp = (torch.full((blocks, B, Hk, D), 3.0, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.full((blocks, Hk), 0.7, device="cuda") for _ in range(2))
    pos = torch.full((n,), ROWS, dtype=torch.int32, device="cuda")
    pos[-1] = 0
    slots = torch.arange(n, device="cuda")
    table = ref.table64(ROWS, D, dev="cuda")
    pkv.kv_append_rope_q8(kp, vp, ks, vs, k, v, slots, pos, table)
    assert _clean() == _lib.DEVERR_POSITION
    last = (n - 1) // B
    for sc, pool in ((ks, kp), (vs, vp)):
        assert (sc[:last] == 0.7).all() and (pool[:last].float() == 3.0).all()
        assert (pool[last, (n - 1) % B + 1:].float() == 3.0).all()
        assert (pool[last, (n - 1) % B].float() != 3.0).any()


def test_a_row_again_behind_left_out_tokens_is_flagged():
    """A token that goes back in its block is not appended, whatever stands between."""
    _clean()
    Hk, D, B = 1, 64, 16
    gen = torch.Generator().manual_seed(43)
    slots = [16, 17] + [-1] * 50 + [17, 18] + [-1] * 300 + [32]
    x = torch.randn(len(slots), Hk, D, generator=gen).to(BF)
    kp, vp = (torch.zeros(4, B, Hk, D, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.ones(4, Hk, device="cuda") for _ in range(2))
    pkv.kv_append_rope_q8(kp, vp, ks, vs, x.cuda(), x.cuda(), torch.tensor(slots).cuda())
    assert _clean() == _lib.DEVERR_SLOT
    keep = [0, 1, len(slots) - 1]
    zero = torch.zeros(3, Hk, D, dtype=torch.float64)
    w = ref.append_q8(torch.zeros(4, B, Hk, D, dtype=torch.float64),
                      torch.ones(4, Hk, dtype=torch.float64), x[keep].double(), zero, [16, 17, 32])
    assert torch.equal(vp.cpu().double(), w[0]) and torch.equal(vs.cpu().double(), w[1])


def test_padding_behind_and_ahead():
    """A short batch in a long padded call, and in its middle."""
    Hk, D, B, n = 2, 128, 32, 5
    gen = torch.Generator().manual_seed(44)
    x = torch.randn(n, Hk, D, generator=gen).to(BF)
    table = ref.table64(64, D, dev="cuda")
    slots, pos = torch.tensor([3, 4, 5, 70, 71]), torch.arange(5, dtype=torch.int32)
    want = None
    for ahead, behind in ((0, 0), (0, 3000), (3000, 0), (511, 700), (90, 100), (0, 9000)):
        T = ahead + n + behind
        k = torch.full((T, Hk, D), 1e4).to(BF)
        k[ahead:ahead + n] = x
        s, p = torch.full((T,), -1), torch.full((T,), 1 << 30, dtype=torch.int32)
        s[ahead:ahead + n], p[ahead:ahead + n] = slots, pos
        kp, vp = (torch.zeros(3, B, Hk, D, device="cuda").to(E4) for _ in range(2))
        ks, vs = (torch.full((3, Hk), 2.0 ** -9, device="cuda") for _ in range(2))
        pkv.kv_append_rope_q8(kp, vp, ks, vs, k.cuda(), k.cuda(), s.cuda(), p.cuda(), table)
        assert _clean() == 0
        got = [y.view(torch.uint8).clone() for y in (kp, vp, ks, vs)]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (ahead, behind)

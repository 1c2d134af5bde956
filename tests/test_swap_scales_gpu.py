"""Copies of an 8-bit cache's scales, of any number of kv heads, and the serving loop's
forks with one, two, three and six of them."""
import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from paged_kv_decode_26_gb300 import _lib
from tests import test_q8_loop_gpu as loop

pytestmark = pytest.mark.gpu


def _clean():
    torch.cuda.synchronize()
    return pkv.device_errors(clear=True)


@pytest.mark.parametrize("Hk", [1, 2, 3, 4, 5, 6, 7, 9, 12, 33])
@pytest.mark.parametrize("n", [1, 30, 3000])
@pytest.mark.parametrize("pinned", [False, True])
def test_scales_of_any_number_of_heads(Hk, n, pinned):
    _clean()
    g = torch.Generator().manual_seed(51)
    ns, nd = n + 4, 2 * n + 3
    src = [torch.randn(ns, Hk, generator=g) for _ in "kv"]
    dst = [torch.randn(nd, Hk, generator=g) for _ in "kv"]
    pairs = torch.stack([torch.randint(0, ns, (n,), generator=g), torch.randperm(nd, generator=g)[:n]], 1)
    bad = torch.tensor([[-1, 0], [0, -1], [ns, 1], [1, nd], [1 << 40, 2]])
    at = src if pinned else [x.cuda() for x in src]
    if pinned:
        at = [x.pin_memory() for x in at]
    dev = pairs.pin_memory() if pinned else pairs.cuda()
    want = [d.clone() for d in dst]
    for w, s in zip(want, src):
        w[pairs[:, 1]] = s[pairs[:, 0]]
    got = [d.cuda() for d in dst]
    pkv.swap_blocks_kv(*got, *at, dev)
    assert _clean() == 0
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
    one = dst[0].cuda()
    pkv.swap_blocks(one, at[0], dev)
    assert _clean() == 0
    assert torch.equal(one.cpu(), want[0])
    pkv.swap_blocks_kv(*got, *at, bad.cuda())
    assert _clean() == _lib.DEVERR_PAIR
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


def test_within_one_pool_on_a_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(52)
    sc = torch.randn(40, 3, generator=g)
    pairs = torch.tensor([[0, 20], [1, 21], [39, 5]]).cuda()
    want = sc.clone()
    want[[20, 21, 5]] = want[[0, 1, 39]]
    a, b = sc.cuda(), sc.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    pkv.swap_blocks(a, a, pairs, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.swap_blocks_kv(b, b.clone(), b, b.clone(), pairs)
    graph.replay()
    assert _clean() == 0
    assert torch.equal(a.cpu(), want) and torch.equal(b.cpu(), want)


def test_offsets_beyond_32_bits():
    n = (1 << 31) // 3 + 1000                      # rows of three floats: beyond 2^31 elements
    sc = torch.zeros(n, 3, device="cuda")
    sc[:2] = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]])
    pkv.swap_blocks(sc, sc, torch.tensor([[0, n - 1], [1, n - 7]]).cuda())
    assert _clean() == 0
    assert sc[n - 1].tolist() == [1, 2, 3] and sc[n - 7].tolist() == [4, 5, 6]
    assert sc[2:n - 7].abs().max() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.uint8, torch.float64])
def test_other_types_of_odd_size_are_refused(dtype):
    x = torch.zeros(4, 3, dtype=dtype, device="cuda")
    with pytest.raises(pkv.PagedKVError):
        pkv.swap_blocks(x, x, torch.zeros(1, 2, dtype=torch.int64, device="cuda"))
    assert _clean() == 0


@pytest.mark.parametrize("H,Hk,D,B,dtype", [
    (1, 1, 128, 16, torch.bfloat16), (8, 2, 64, 16, torch.float16), (3, 3, 64, 32, torch.bfloat16),
    (6, 6, 64, 16, torch.float16)])
def test_serving_loop_of_few_heads(H, Hk, D, B, dtype):
    loop.test_serving_loop(H, Hk, D, B, dtype, D, False)

"""The cache operators on two streams at once, and as graphs replayed side by
side: results equal those of calls made alone, bit for bit.  Also the smallest
prompts and decodes of every head layout."""

import pytest
import torch

import paged_kv_decode_26_gb300 as pkv
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _jobs(out_dtype):
    """Closures that each run one operator on tensors of their own, and the
    tensors they write."""
    jobs = []
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    lens = [900, 1, 130, 700, 64, 513]
    starts = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
    q, k, v = rnd(sum(lens), 32, 128), rnd(sum(lens), 8, 128), rnd(sum(lens), 8, 128)
    po = torch.zeros(sum(lens), 32, 128, dtype=out_dtype, device="cuda")
    jobs.append((lambda: pkv.attn_prompt(po, q, k, v, starts, 0.09, 900), [po]))
    for prefix in (256, 1024):
        c = ref.paged([prefix + 10 + 7 * i for i in range(12)], 16, 8, 128, BF, prefix,
                      shared=([0, 6, 12], [prefix, prefix]))
        dq = rnd(12, 32, 128)
        so = torch.zeros(12, 32, 128, dtype=out_dtype, device="cuda")
        gs, pl, L = _ints([0, 6, 12]), _ints([prefix, prefix]), prefix + 100
        jobs.append((lambda c=c, dq=dq, so=so, gs=gs, pl=pl, L=L, prefix=prefix:
                     pkv.paged_attn_decode_shared(so, dq, c["k_pool"], c["v_pool"], c["tables"],
                                                  c["lens"], gs, pl, 0.09, L, 6, prefix), [so]))
        w = torch.zeros(12, L, device="cuda")
        wo = torch.zeros(12, 32, 128, dtype=out_dtype, device="cuda")

        def weights(c=c, dq=dq, wo=wo, w=w, L=L):
            w.zero_()
            pkv.paged_attn_decode_weights(wo, dq, c["k_pool"], c["v_pool"], c["tables"], c["lens"],
                                          w, 0.09, L)
        jobs.append((weights, [wo, w]))
    return jobs


@pytest.fixture
def once():
    pkv.set_tuning(shared_prefix=1)
    yield
    pkv.reset_tuning()


@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_streams_side_by_side(once, out_dtype):
    jobs = _jobs(out_dtype)
    want = []
    for run, outs in jobs:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _, outs in jobs:
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for (run, _), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    for (_, outs), exp in zip(jobs, want):
        for o, e in zip(outs, exp):
            assert torch.equal(o, e)


def test_graphs_side_by_side(once):
    jobs = _jobs(BF)
    want, graphs = [], []
    for run, outs in jobs:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert pkv.device_errors(clear=True) == 0
    for (_, outs), exp in zip(jobs, want):
        for o, e in zip(outs, exp):
            assert torch.equal(o, e)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("Hk", [1, 2, 5, 8])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_one_token_of_every_head_layout(G, Hk, out_dtype):
    """A prompt, and decodes, of one token: the output is V itself."""
    H, D = G * Hk, 64
    g = torch.Generator().manual_seed(Hk)
    q, k, v = (torch.randn(1, h, D, generator=g).to(BF).cuda() for h in (H, Hk, Hk))
    want = v.repeat_interleave(G, 1).to(out_dtype)
    out = torch.empty(1, H, D, dtype=out_dtype, device="cuda")
    pkv.attn_prompt(out, q, k, v, _ints([0, 1]), 0.1, 1)
    assert torch.equal(out, want)
    pool_k, pool_v = (torch.full((1, 16, Hk, D), float("nan"), dtype=BF, device="cuda")
                      for _ in range(2))
    pool_k[0, 0], pool_v[0, 0] = k[0], v[0]
    w = torch.zeros(1, 1, device="cuda")
    out.zero_()
    pkv.paged_attn_decode_weights(out, q, pool_k, pool_v, _ints([[0]]), _ints([1]), w, 0.1, 1)
    assert torch.equal(out, want) and float(w) == H
    out.zero_()
    pkv.paged_attn_decode_shared(out, q, pool_k, pool_v, _ints([[0]]), _ints([1]), _ints([0, 1]),
                                 _ints([0]), 0.1, 1, 1, 0)
    assert torch.equal(out, want)
    assert pkv.device_errors(clear=True) == 0

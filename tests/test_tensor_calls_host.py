"""The native part of the binding without a device: what it refuses before any call."""
import pytest
import torch

from paged_kv_decode_26_gb300 import build


@pytest.fixture(scope="module")
def pkv():
    build.build()
    import paged_kv_decode_26_gb300 as pkv
    return pkv


def test_tensors_of_the_host_are_refused(pkv):
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    p8, sc = pool.to(torch.float8_e4m3fn), torch.ones(4, 2)
    slots, ints = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    tables = torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.kv_append_rope(pool, pool.clone(), k, k, slots)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.kv_append_rope_q8(p8, p8.clone(), sc, sc.clone(), k, k, slots)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.paged_attn_decode_q8(k.clone(), k, p8, p8, sc, sc, tables, ints, 0.1, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.paged_attn_multi_query_q8(k.clone(), k, torch.zeros(4, dtype=torch.int32), p8, p8, sc, sc,
                                      tables, ints, 0.1, 1, 64)


def test_what_is_no_tensor(pkv):
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in (lambda: pkv.kv_append_rope(None, k, k, k, k),
                lambda: pkv.kv_append_rope(k, k, k, k, 5),
                lambda: pkv.paged_attn_decode_q8(k, "q", k, k, k, k, k, k, 0.1, 64)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    from paged_kv_decode_26_gb300 import _lib
    for name in ("kv_append_rope", "kv_append_rope_q8", "paged_attn_decode_q8",
                 "paged_attn_multi_query_q8"):
        with pytest.raises(ValueError, match="arguments"):
            getattr(_lib.calls(), name)(k)

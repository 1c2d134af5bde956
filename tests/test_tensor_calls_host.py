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


_WITHOUT_STORAGE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from paged_kv_decode_26_gb300 import _lib
c = _lib.calls()
F8, F32, I32 = torch.float8_e4m3fn, torch.float32, torch.int32
with FakeTensorMode():
    def e(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    k, slots, start = e(3, 2, 64), e(3, dtype=torch.int64), e(4, dtype=I32)
    p16 = [e(4, 16, 2, 64) for _ in "kv"]
    p8 = [e(4, 16, 2, 64, dtype=F8) for _ in "kv"] + [e(4, 2, dtype=F32) for _ in "kv"]
    rest = (None, None, None, None, None, False, 0)
    held = (e(3, 4, dtype=I32), e(3, dtype=I32), 0.1)
    for call in (lambda x: c.kv_append_rope(*p16, x, k, slots, *rest),
                 lambda x: c.kv_append_rope_q8(*p8, k, x, slots, *rest),
                 lambda x: c.paged_attn_decode_q8(k, x, *p8, *held, 64, None, 0),
                 lambda x: c.paged_attn_multi_query_q8(k, x, start, *p8, *held, 1, 64, None, 0)):
        try:
            torch.vmap(lambda x: call(x) and x)(e(5, 3, 2, 64))
        except RuntimeError:
            print("raised", flush=True)
"""


def test_a_tensor_without_storage_raises(pkv, tmp_path):
    """vmap's tensors have no data pointer: an exception, and the interpreter lives.  (In
    a process of its own, whose tensors only say that they are on a GPU.)"""
    import os
    import subprocess
    import sys
    src, shim = tmp_path / "device.cpp", tmp_path / "device.so"
    src.write_text("namespace c10 { namespace cuda { signed char current_device() { return 0; } } }")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(shim), str(src)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, LD_PRELOAD=str(shim), PYTHONPATH=root)
    got = subprocess.run([sys.executable, "-c", _WITHOUT_STORAGE], env=env, cwd=root,
                         capture_output=True, text=True, timeout=600)
    assert got.returncode == 0, got.stderr[-500:]
    assert got.stdout.split() == ["raised"] * 4

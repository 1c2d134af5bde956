"""When the library and the binding's extension are built anew, and what a torch without
CUDA leaves out.  Nothing is compiled here but what is missing."""
import os
import sys

import pytest
import torch

from paged_kv_decode_26_gb300 import _lib, build


@pytest.fixture
def steps(monkeypatch):
    """The build's steps as they are taken, none of them done."""
    build.build()
    taken = []
    monkeypatch.setattr(build, "_compile", lambda src, v: taken.append("compile") or "o")
    monkeypatch.setattr(build, "_compile_calls", lambda: taken.append("compile extension") or "o")
    monkeypatch.setattr(build, "_link_calls", lambda obj: taken.append("link extension"))

    def run(*a, **k):
        raise AssertionError("a library linked")

    monkeypatch.setattr(build.subprocess, "run", run)
    return taken


def test_nothing_to_do(steps):
    assert build.up_to_date()
    assert build.build() == build.LIB and steps == []


def test_another_torch_builds_the_extension_anew(steps, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not build.up_to_date()
    build.build()
    assert steps == ["compile extension", "link extension"]


def test_an_extension_of_unknown_origin_is_built_anew(steps, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "none"))
    assert not build.up_to_date()
    build.build()
    assert steps == ["compile extension", "link extension"]


def test_its_source_builds_the_extension_alone(steps, monkeypatch, tmp_path):
    src = tmp_path / "tensor_calls.cpp"
    src.write_text("")
    future = os.path.getmtime(build.CALLS) + 100
    os.utime(src, (future, future))
    monkeypatch.setattr(build, "CALLS_SRC", str(src))
    build.build()
    assert steps == ["compile extension", "link extension"]


def test_without_cuda_in_torch_the_library_is_all(steps, monkeypatch, tmp_path):
    monkeypatch.setattr(torch.version, "cuda", None)
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "none.so"))
    assert build.up_to_date()
    assert build.build() == build.LIB and steps == []


def test_calls_without_the_extension_say_so(monkeypatch):
    build.build()
    monkeypatch.setattr(_lib, "_calls", None)
    monkeypatch.setitem(sys.modules, "paged_kv_decode_26_gb300._tensor_calls", None)
    import paged_kv_decode_26_gb300 as package
    monkeypatch.delattr(package, "_tensor_calls", raising=False)
    with pytest.raises(RuntimeError, match="CUDA build of torch"):
        _lib.calls()

"""Build libpagedkv.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_tensor_calls.so (the part of the binding that is native) with g++.

Each translation unit compiles in parallel to an object under _build/, then
nvcc links the shared library next to this file, and g++ the extension against
it.  Rebuilds the library only when a source or header is newer, and the extension
only then or when torch or Python are others than it was built with.  The library needs
nvcc alone: without a CUDA build of torch there is no extension, and the calls that go
through it say so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
CALLS_SRC = os.path.join(HERE, "csrc_py", "tensor_calls.cpp")
CALLS = os.path.join(HERE, "_tensor_calls.so")
CALLS_STAMP = os.path.join(BUILD, "tensor_calls.built_with")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--use_fast_math", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.inc")) +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    """Whether the library and, where torch has CUDA, the extension are."""
    return _lib_up_to_date() and (_calls_stamp() is None or _calls_up_to_date())


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _calls_stamp() -> str | None:
    """What the extension's binary depends on besides its source; None without a CUDA
    build of torch."""
    try:
        import torch
    except ImportError:
        return None
    if torch.version.cuda is None:
        return None
    return "\n".join([torch.__version__, torch.version.cuda, os.path.dirname(torch.__file__),
                      str(int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))),
                      str(sysconfig.get_config_var("SOABI"))])


def _calls_up_to_date() -> bool:
    try:
        with open(CALLS_STAMP) as f:
            built = f.read()
    except OSError:
        return False
    return built == _calls_stamp() and _newer(CALLS, [CALLS_SRC, os.path.join(INCLUDE, "pagedkv.h"),
                                                      os.path.abspath(__file__)])


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas:
        print(res.stderr)
    return obj


def _compile_calls() -> str:
    """The extension's object (its headers are torch's and Python's)."""
    import torch
    top = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(BUILD, "tensor_calls.cpp.o")
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", top,
           "-I", os.path.join(top, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", cuda, "-c", CALLS_SRC, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libpagedkv.so", "-L", libs,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_STAMP, "w") as f:
        f.write(_calls_stamp())


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    lib = force or not _lib_up_to_date()
    calls = _calls_stamp() is not None and (force or not _calls_up_to_date())
    if not (lib or calls):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources() if lib else []
    jobs = jobs or min(len(srcs) + 1, os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls_obj = ex.submit(_compile_calls) if calls else None
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if lib:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    if calls:
        _link_calls(calls_obj.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))

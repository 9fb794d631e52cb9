"""Build the CUDA library libdspark.so in-tree for sm_103a (GB300).

Each translation unit compiles in parallel with nvcc; the objects link into
one shared library whose exported symbols are exactly the C ABI of
include/dspark.h.  Beside it g++ compiles the Python calls of the target-pass
operators (bind.cpp, against the installed PyTorch's headers) into a module that
links to the library; the library does not need the module.  Outputs go to
speculative_decoding_drafter_markov_gb300/_build/.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libdspark.so")
SOURCES = ["abi.cu", "attn.cu", "attn4_mma.cu", "attn4_tc.cu", "attn_f32.cu", "attn_tc.cu", "cache4.cu", "diag.cu", "draft.cu", "draft_tc.cu", "gemm_tc.cu", "paged.cu", "rope.cu", "rules.cu",
           "sched.cu", "sts.cu", "train_loss.cu", "verify.cu", "verify_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
TU_FLAGS = {}
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the DSpark CUDA library cannot be built")


HEADER = os.path.join(ROOT, "include", "dspark.h")
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")


def _current(out, deps) -> bool:
    return os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(f) for f in deps)


def _library_deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "bind.cpp"] + [HEADER]


def bind_path() -> str:
    """The module's file, named by what its machine code depends on: PyTorch's C++
    interface and Python's.  Another PyTorch finds no module of its name and builds one."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(OUT, f"_dspark_bind.torch{torch.__version__}.abi{abi}.{sysconfig.get_config_var('SOABI')}.so")


def _compile_bind(obj: str) -> None:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"], "/usr/local/cuda/include")),
           "-c", BIND_SOURCE, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{res.stderr}")


def _link_bind(obj: str, out: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + f".{os.getpid()}.tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", OUT, "-l:libdspark.so", "-Wl,-rpath,$ORIGIN",
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{res.stderr}")
    os.replace(tmp, out)


def build_bind(force: bool = False, library=None) -> str:
    """The module of the target-pass calls (bind.cpp), for the Python and the PyTorch
    that run.  `library` waits for the library, which is built if it is not given."""
    out = bind_path()
    if not force and _current(out, [BIND_SOURCE, HEADER]):
        return out
    os.makedirs(OUT, exist_ok=True)
    obj = os.path.join(OUT, f"bind.{os.getpid()}.o")
    try:
        _compile_bind(obj)
        (library or build)()
        _link_bind(obj, out)
    finally:
        if os.path.exists(obj):
            os.remove(obj)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    """The library."""
    os.makedirs(OUT, exist_ok=True)
    if not force and _current(LIB, _library_deps()):
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT, src.replace(".cu", ".o"))
        extra = TU_FLAGS.get(src, [])
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
        if verbose and res.stderr:
            sys.stderr.write(res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    res = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_all(force: bool = False, verbose: bool = False) -> str:
    """The library and the module, compiled side by side."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=2) as ex:
        library = ex.submit(build, force, verbose)
        bind = ex.submit(build_bind, force, library.result)
        path = library.result()
        bind.result()
    return path


if __name__ == "__main__":
    print(build_all(force="--force" in sys.argv, verbose="-v" in sys.argv))

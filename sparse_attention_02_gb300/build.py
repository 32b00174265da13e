"""Build libdsa.so (sm_103a) in-tree with nvcc.

Each translation unit under csrc/ compiles in parallel to an object file, then
one link step makes ``sparse_attention_02_gb300/libdsa.so``; the host compiler
makes ``_fastcall.so``, the native part of the Python binding.  Run as a script
or call ``build()``.  The library needs the CUDA toolkit alone (no cmake).  The
extension takes a C++ compiler, Python's headers and PyTorch's (torch itself is not
imported); without the headers it is left out, and the binding does without it.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_objs")
LIB = os.path.join(HERE, "libdsa.so")
FAST = os.path.join(HERE, "_fastcall.so")
FAST_KEY = os.path.join(HERE, "_fastcall.key")  # what FAST was built for and from
SOURCES = ["api.cu", "quantize.cu", "rmsnorm.cu", "rmsnorm_backward.cu", "rope.cu", "indexer.cu", "topk.cu", "indexer_topk.cu", "warmup.cu",
           "sparse_mla.cu", "dense_mla.cu", "prefill_host.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                   "-I", os.path.join(HERE, "..", "include"), *extra]


def _compile(src: str, extra=()) -> str:
    obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    deps = [path] + [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".cuh", ".h"))]
    deps.append(os.path.join(HERE, "..", "include", "dsa.h"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps):
        return obj
    cmd = [nvcc(), "-c", path, "-o", obj + ".tmp"] + _flags(extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj


def _torch_root():
    torch = importlib.util.find_spec("torch")
    return None if torch is None else list(torch.submodule_search_locations)[0]


def _digest(*paths) -> str:
    h = hashlib.sha256()
    for p in paths:
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def fastcall_abi() -> str:
    """What ``_fastcall.so`` is compiled against and finds at run time: this interpreter's ABI and this PyTorch."""
    root = _torch_root()
    return f"{sysconfig.get_config_var('SOABI')} {root} {_digest(os.path.join(root, 'version.py'))}"


def fastcall_built_for() -> str:
    """The same of the ``_fastcall.so`` that is there; empty where it does not say."""
    try:
        with open(FAST_KEY) as f:
            return f.readline().rstrip("\n")
    except OSError:
        return ""


def _build_fastcall():
    src, hdr = os.path.join(CSRC, "fastcall.cpp"), os.path.join(HERE, "..", "include", "dsa.h")
    root = _torch_root()
    if root is None:  # no binding without it; the library stands alone
        return
    for need in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h")):
        if not os.path.exists(need):
            warnings.warn(f"{need} is missing: _fastcall.so is not built", RuntimeWarning)
            return
    cxx = os.environ.get("CXX", "g++")
    key = f"{fastcall_abi()}\n{cxx} {_digest(src, hdr, os.path.abspath(__file__))}\n"
    if os.path.exists(FAST) and os.path.exists(FAST_KEY):
        with open(FAST_KEY) as f:
            if f.read() == key:
                return
    tmp = FAST + f".tmp{os.getpid()}"
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), src, "-o", tmp, "-L", lib, "-lc10", "-ltorch_cpu",
           "-ltorch_python", f"-Wl,-rpath,{lib}", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for fastcall.cpp:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(FAST_KEY):  # until the new one is written, the extension counts as built for nothing
        os.remove(FAST_KEY)
    os.replace(tmp, FAST)
    with open(tmp, "w") as f:
        f.write(key)
    os.replace(tmp, FAST_KEY)


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fast = ex.submit(_build_fastcall)
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
        fast.result()
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), "-shared", "-o", tmp, *objs] + ARCH + ["-Xcompiler", "-fPIC", "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])

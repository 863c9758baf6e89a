"""Build the pkv CUDA library (libpkv.so) in-tree for sm_103a.

Each translation unit is compiled in parallel with nvcc, then linked into one
shared library next to this file. Beside it the CPython module _pkv_call
(csrc/host/pkv_call.cpp, the argument checks of the serving calls) is built with
the host compiler against the installed torch, under a name that says which
Python and torch that was. Rebuilds only when a source is newer than what it
makes.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import re
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIBRARY = os.path.join(HERE, "libpkv.so")
CALL_SOURCE = os.path.join(CSRC, "host", "pkv_call.cpp")
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-ffp-contract=off"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    # CUDA translation units and host-only C++ (the page scheduler), all through nvcc
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIBRARY):
        return False
    t = os.path.getmtime(LIBRARY)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def call_module() -> str:
    """Where the CPython module for the Python and torch that run this is. It is
    bound to torch's C++ interface, so every torch (its version, the commit it
    was built from, its C++ ABI) has a file of its own and none is loaded into another."""
    import torch
    tag = (f"{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}-{str(torch.version.git_version)[:8]}"
           f"-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}")
    return os.path.join(HERE, "_pkv_call." + re.sub(r"[^\w.+-]", "_", tag) + ".so")


def build_call(force: bool = False) -> str:
    """The CPython module, against the Python and torch that run this."""
    module = call_module()
    inputs = [CALL_SOURCE, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(module) and all(os.path.getmtime(f) <= os.path.getmtime(module) for f in inputs):
        return module

    import torch
    root = os.path.dirname(torch.__file__)
    include = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    tmp = module + f".{os.getpid()}.tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include),
           CALL_SOURCE, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiler failed for {CALL_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, module)
    return module


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        build_call()
        return LIBRARY
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + ARCH + (extra_flags or []) + ["-I", INCLUDE]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + f".{os.getpid()}.o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources()) + 1) as ex:
        module = ex.submit(build_call, force)
        objs = list(ex.map(compile_one, sources()))
        module.result()
    tmp = LIBRARY + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    for o in objs:
        os.remove(o)
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, extra_flags=sys.argv[1:]))

"""In-tree build of libhs.so (the C ABI of include/hs.h) for sm_103a with nvcc, and of the
torch binding of the page calls (host code only).

Each CUDA translation unit is compiled in parallel, then linked into a shared
library next to this file. Nothing is installed into site-packages.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhs.so")
TORCH_LIB = os.path.join(HERE, "_hs_torch.so")  # the compiled part of the Python binding
TORCH_SOURCE = os.path.join(CSRC, "hs_torch.cpp")
SOURCES = ["hs_api.cu", "hs_kernels.cu", "hs_noalloc.cu", "hs_consume.cu", "hs_attend.cu", "hs_pool.cu",
           "hs_page.cu", "hs_page_attend.cu"]
HEADERS = [os.path.join(CSRC, "hs_internal.h"), os.path.join(CSRC, "hs_page.h"), os.path.join(CSRC, "hs_once.h"),
           os.path.join(ROOT, "include", "hs.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-v",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_command(obj: str) -> list[str]:
    """The host compiler's command for the torch binding (headers of the torch that runs)."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(cuda or "/usr/local/cuda", "include")]
    return (["g++", "-O2", "-fPIC", "-std=c++17", "-I", os.path.join(ROOT, "include"),
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
            + [x for d in dirs for x in ("-isystem", d)] + ["-c", TORCH_SOURCE, "-o", obj])


def _link_torch(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    subprocess.check_call(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libhs.so", "-Wl,-rpath,$ORIGIN", "-L", libs,
                           f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, TORCH_LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libhs.so and the torch binding if any source or header changed;
    returns the path of libhs.so."""
    os.makedirs(OBJDIR, exist_ok=True)
    objs, procs = [], []
    tobj = os.path.join(OBJDIR, "hs_torch.o")
    if force or _stale(tobj, [TORCH_SOURCE] + HEADERS):
        cmd, log = _torch_command(tobj), tobj + ".log"
        procs.append((cmd, log, subprocess.Popen(cmd, stdout=open(log, "w"), stderr=subprocess.STDOUT)))
    for src in SOURCES:
        sp = os.path.join(CSRC, src)
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [sp] + HEADERS):
            log = obj + ".log"
            cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", sp, "-o", obj]
            procs.append((cmd, log, subprocess.Popen(cmd, stdout=open(log, "w"), stderr=subprocess.STDOUT)))
    for cmd, log, p in procs:
        rc = p.wait()
        text = open(log).read()
        if verbose or rc != 0:
            sys.stderr.write(text)
        if rc != 0:
            raise RuntimeError(f"compilation failed ({rc}): {' '.join(cmd)}\n{text}")
    if force or procs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    if force or _stale(TORCH_LIB, [tobj]):
        _link_torch(tobj)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)

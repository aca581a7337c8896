"""In-tree build of libhs.so (the C ABI of include/hs.h) for sm_103a with nvcc, and of the
torch binding of the page calls (host code only).

Each CUDA translation unit is compiled in parallel, then linked into a shared
library next to this file. Nothing is installed into site-packages.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

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


def _torch_dir() -> str:
    """Where the torch that would be imported is (without importing it)."""
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _torch_command(obj: str) -> list[str]:
    """The host compiler's command for the torch binding (headers of the torch that runs), but
    for the flag of its C++ ABI."""
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(cuda or "/usr/local/cuda", "include")]
    return (["g++", "-O2", "-fPIC", "-std=c++17", "-I", os.path.join(ROOT, "include")]
            + [x for d in dirs for x in ("-isystem", d)] + ["-c", TORCH_SOURCE, "-o", obj])


def _torch_stamp(cmd: list[str]) -> str:
    """What the binding is compiled with and against, besides its sources: the command, the
    Python, and the torch, by its library's size and time (its version and ABI with it)."""
    lib = os.stat(os.path.join(_torch_dir(), "lib", "libtorch_python.so"))
    return "\n".join([" ".join(cmd), sys.version, f"{lib.st_size} {lib.st_mtime_ns}"])


def _link_torch(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    subprocess.check_call(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libhs.so", "-Wl,-rpath,$ORIGIN", "-L", libs,
                           f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, TORCH_LIB)


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libhs.so and the torch binding if any source or header changed, the
    binding also for another torch or Python (and not at all where torch is not installed);
    returns the path of libhs.so."""
    os.makedirs(OBJDIR, exist_ok=True)
    objs, procs = [], []
    tobj = os.path.join(OBJDIR, "hs_torch.o")
    with_torch = importlib.util.find_spec("torch") is not None  # else the library alone: the page calls from Python need it
    compile_torch = False
    if with_torch:
        tcmd, tstamp = _torch_command(tobj), tobj + ".stamp"
        stamp = _torch_stamp(tcmd)
        compile_torch = force or _stale(tobj, [TORCH_SOURCE] + HEADERS) or _read(tstamp) != stamp
    if compile_torch:
        import torch
        cmd, log = tcmd + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"], tobj + ".log"
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
    if with_torch and (compile_torch or _stale(TORCH_LIB, [tobj])):
        _link_torch(tobj)
        with open(tstamp, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)

"""When the torch binding is compiled again."""
import os
import subprocess
import sys

import pytest

import hierarchical_kv_cache_swap_gb300 as hs
from hierarchical_kv_cache_swap_gb300 import _nvcc


class Compilers:
    """Stands in for subprocess.Popen: notes the commands and compiles nothing."""

    def __init__(self):
        self.sources = []

    def __call__(self, cmd, stdout=None, **_):
        self.sources.append(next(os.path.basename(x) for x in cmd if x.endswith((".cu", ".cpp"))))
        stdout.close()
        return self

    def wait(self):
        return 0


@pytest.fixture
def compilers(monkeypatch):
    hs.build()
    kept = {}
    for name in os.listdir(_nvcc.OBJDIR):
        if not name.endswith(".o"):
            with open(os.path.join(_nvcc.OBJDIR, name)) as f:
                kept[name] = f.read()
    fake = Compilers()
    monkeypatch.setattr(_nvcc.subprocess, "Popen", fake)
    monkeypatch.setattr(_nvcc.subprocess, "check_call", lambda *a, **k: 0)
    monkeypatch.setattr(_nvcc.os, "replace", lambda *a: None)
    yield fake
    for name, text in kept.items():
        with open(os.path.join(_nvcc.OBJDIR, name), "w") as f:
            f.write(text)


def test_nothing_is_compiled_twice(compilers):
    hs.build()
    assert compilers.sources == []


@pytest.mark.parametrize("what", ["python", "torch", "command"])
def test_the_binding_follows_the_torch_and_python_it_is_compiled_against(compilers, monkeypatch, what):
    if what == "python":
        monkeypatch.setattr(_nvcc.sys, "version", "another")
    elif what == "torch":  # the same place, other files
        stat = os.stat
        monkeypatch.setattr(_nvcc.os, "stat", lambda p, *a, **k: stat(__file__) if str(p).endswith("libtorch_python.so") else stat(p, *a, **k))
    else:
        monkeypatch.setenv("CUDA_HOME", "/nowhere")
        monkeypatch.setattr(_nvcc, "nvcc", lambda: "/elsewhere/bin/nvcc")
    hs.build()
    assert compilers.sources == ["hs_torch.cpp"]
    hs.build()
    assert compilers.sources == ["hs_torch.cpp"]  # and once


def test_the_library_builds_where_torch_is_not_installed(compilers, monkeypatch):
    find = _nvcc.importlib.util.find_spec
    monkeypatch.setattr(_nvcc.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert hs.build(force=True) == _nvcc.LIB
    assert sorted(compilers.sources) == sorted(_nvcc.SOURCES)


WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None  # as if it were not installed
sys.path.insert(0, sys.argv[1])
import hierarchical_kv_cache_swap_gb300 as hs
hs.build()
assert hs.PageShape(16, 8, 128).bytes == 18432
try:
    hs.write_tokens((16, 8, 128), None, None, None, None)
except ImportError as e:
    print("page calls:", e)
"""


def test_the_library_is_usable_where_torch_is_not_installed():
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH, _nvcc.ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "page calls: " in r.stdout, r.stdout + r.stderr

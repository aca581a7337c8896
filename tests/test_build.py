"""When the torch binding is compiled again."""
import os

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

"""What a wait for the last kernel of a call covers, read from the sources: a programmatic
dependent waits for the grid directly ahead of it and for no earlier one, so every kernel of a
chain of them has to wait for its own predecessor before it ends."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_cache_swap_gb300", "csrc")
WAIT = re.compile(r"(?:if \(([^;{}]*?)\)\s*)?(?:pdl_wait_prerequisites\(\)|asm volatile\(\"griddepcontrol\.wait;\" ::: \"memory\"\));")


def kernels():
    """{name: body} of every kernel in a source file that launches programmatic dependents."""
    found = {}
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        if "cudaLaunchAttributeProgrammaticStreamSerialization" not in text:
            continue
        for m in re.finditer(r"__global__ void __launch_bounds__\([^)]*\)\s*(\w+)\s*\([^{;]*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            found[m.group(1)] = text[m.end():i]
    return found


def conditions(body):
    """The conditions of a kernel's own waits (None: always)."""
    return [m.group(1) for m in WAIT.finditer(body)]


def test_the_kernels_are_found():
    assert set(kernels()) == {"resolve_kernel", "gather_kernel", "write_kernel", "read_kernel", "attend_pages_kernel"}


@pytest.mark.parametrize("name", ["gather_kernel", "write_kernel", "read_kernel", "attend_pages_kernel"])
def test_dependents_always_wait_and_leave_no_earlier(name):
    body = kernels()[name]
    assert conditions(body) == [None]
    assert not re.search(r"\breturn\b", re.split(WAIT, body)[0])


@pytest.mark.parametrize("chunks", [1, 2, 3, 7])
def test_the_last_fetch_of_a_call_ends_after_all_the_others(chunks):
    """A call of several chunks: resolution, fetch, resolution, fetch, ... and a successor that
    waits for the last fetch. The first resolution waits before its work, the later ones do not."""
    asked = conditions(kernels()["resolve_kernel"])
    waits = {1: "wait" in asked or None in asked, 0: "!wait && blockIdx.x == 0" in asked or "!wait" in asked or None in asked}
    done, complete = set(), set()  # of the grid so far; grids whose end its end implies
    for i in range(chunks):
        for kind in ("resolve", "fetch"):
            own = waits[1 if i == 0 else 0] if kind == "resolve" else conditions(kernels()["gather_kernel"]) == [None]
            done = {(kind, i)} | (done if own else set())
            complete.add((kind, i))
    assert done == complete

"""The limit of the latent kernels' waits, without a GPU."""
import os
import re
import threading

import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()
    yield
    hs.set_latent_waits()


def test_the_limit_and_the_flags_are_checked():
    for bad in (0, 999, 10_000_000_001, -1):
        with pytest.raises(hs.HsError, match="outside"):
            hs.set_latent_waits(bad)
    for good in (1000, 10_000_000_000):
        hs.set_latent_waits(good, stall=True)
    lib = hs.load_library()
    for flags in (1, 4, 3):
        assert lib.hs_set_latent_waits(1000, flags) == hs.HS_ERR_INVALID
        assert "unknown flags" in hs.last_error()
    hs.set_latent_waits()


def test_threads_set_their_own():
    got = []
    t = threading.Thread(target=lambda: got.append(hs.load_library().hs_set_latent_waits(1000, 2)))
    t.start()
    t.join()
    assert got == [hs.HS_OK]


def kernel(name, source="hs_absorb.cu", first="const HeadProduct p"):
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_cache_swap_gb300", "csrc")
    with open(os.path.join(csrc, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return re.split(r"__global__ void", text.split(name + "(" + first)[1])[0]


def test_absorbed_queries_leave_what_is_in_flight_alone():
    """After a wait that ran out, a copy or the products may still be at work on the operands' place: their
    end is told by `over`, which the other warps wait for before they write there."""
    body = kernel("absorb_kernel")
    steps = ["mma_commit(&sm->done);", "mma_commit(&sm->over);", "bar_drain(&sm->landed", "bar_arrive(&sm->over)", "bar_wait(&sm->done",
             "bar_drain(&sm->over", "*reinterpret_cast<uint32_t*>(to", "__syncthreads();\n    if (warp == 4)", "tmem_free"]
    assert [body.count(x) for x in steps] == [1] * len(steps)
    assert [body.index(x) for x in steps] == sorted(body.index(x) for x in steps)


def test_expanded_outputs_leave_what_is_in_flight_alone():
    """After a wait that ran out no warp writes a next tile, and none frees the columns, before the products of
    this one have ended: `over` tells, once a tile in any case."""
    loop = kernel("expand_many_kernel").split("for (int k = 0; t0 < p.n;")[1]
    steps = ["mma_commit(&sm->done[group]);", "mma_commit(&sm->over[group]);", "if (__builtin_expect(!ok, 0) && lane == 0) bar_arrive(&sm->over[group]);",
             "bar_wait(&sm->done[group], k & 1", "bar_drain(&sm->over[group], k & 1", "tmem_load16", "tmem_free"]
    assert [loop.count(x) for x in steps] == [1] * len(steps)
    assert [loop.index(x) for x in steps] == sorted(loop.index(x) for x in steps)


def test_the_outputs_call_takes_a_status_word():
    o, up, out = torch.zeros(2, 4, 512), torch.zeros(4, 128, 512, dtype=torch.bfloat16), torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the CPU"):
        hs.expand_outputs(o, up, out, status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="5 arguments"):
        hs._native().expand_outputs(o, up, out, None)
    assert hs._HeadProduct().status is None and hs._HeadProduct._fields_[-1][0] == "status"


def test_each_row_tiles_queries_are_waited_for_at_the_end():
    """The copies of an item's queries are issued a row tile at a time, with a wait between them that may run out:
    what is on its way is noted for each, before it is."""
    body = kernel("prompt_kernel", "hs_prompt.cu", "const PromptAttention A")
    turn = body[body.index("until(&sm->q_free[w], k - 1)"):body.index("&maps.q, 0, q_row")]
    assert turn.count("(w ? asked1 : asked0) = k;") == 1
    assert re.search(r"asked = w \? asked1 : asked0;\s*if \(asked >= 0\) bar_drain\(&sm->q_full\[w\], asked & 1", body)


@pytest.mark.parametrize("name,source,first", [("absorb_kernel", "hs_absorb.cu", "const HeadProduct p"), ("expand_many_kernel", "hs_absorb.cu", "const HeadProduct p"),
                                               ("prompt_kernel", "hs_prompt.cu", "const PromptAttention A")])
def test_what_is_in_flight_is_waited_for_longer_than_it_can_take(name, source, first):
    """However short the limit of a wait: a copy landing behind its CTA's end would land in another's memory."""
    drains = re.findall(r"bar_drain\(([^;]*)\);", kernel(name, source, first))
    assert drains and all(x.endswith("waits.drain") for x in drains)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_cache_swap_gb300", "csrc")
    with open(os.path.join(csrc, "hs_latent.h")) as f:
        text = f.read()
    assert "kLeastDrainNs = 10000000ull" in text and "ns > kLeastDrainNs ? ns : kLeastDrainNs" in text

"""Refusals of the page attention's checks, without a GPU."""
import ctypes
import itertools
import random

import pytest

import hierarchical_kv_cache_swap_gb300 as hs
from tests.test_pages import _attention


@pytest.fixture(scope="module")
def lib():
    hs.build()
    return hs.load_library()


def refused(lib, B, T, H, strides):
    """Whether the call is refused for overlapping rows of o. No request is attended: with B = 0
    nothing is launched, and the batch is put among the query tokens or heads instead."""
    a = _attention(shape=hs._PageShape(16, 1, 128), B=B, q_tokens=T, q_heads=H, o_batch_stride=strides[0],
                   o_token_stride=strides[1], o_head_stride=strides[2])
    rc = lib.hs_attend_pages(None, ctypes.byref(a))
    if rc == hs.HS_ERR_INVALID:
        assert "overlap" in hs.last_error()
    return rc == hs.HS_ERR_INVALID


@pytest.mark.parametrize("T,H,strides", [
    (2, 2, (0, 128, 128)),        # (t0, h1) is (t1, h0)
    (3, 4, (0, 256, 128)),        # (t0, h2) is (t1, h0)
    (2, 8, (0, 1000, 128)),       # (t1, h0) begins inside (t0, h7)
    (2, 8, (0, -1000, 128)),
    (5, 3, (0, 384, 1536)),       # (t4, h0) is (t0, h1)
    (2, 3, (0, 128 * 2**54, 128 * 2**54)),
])
def test_rows_that_meet_through_two_strides_are_refused(lib, T, H, strides):
    assert refused(lib, 0, T, H, strides)


@pytest.mark.parametrize("B,T,H,strides", [(2, 2, 2, (256, 256, 128)), (3, 2, 1, (128, 256, 0)), (2, 2, 2, (384, 256, 128))])
def test_rows_that_meet_through_the_batch_are_refused(lib, B, T, H, strides):
    assert refused(lib, B, T, H, strides)


def test_rows_are_refused_exactly_when_two_of_them_overlap(lib):
    """Random small extents and strides, interleaved ones that no row shares among them."""
    rng = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        T, H = rng.randint(1, 5), rng.randint(1, 6)
        strides = (0, *(rng.choice((-1, 1)) * 8 * rng.choice((rng.randint(0, 120), 16 * rng.randint(1, 8))) for _ in range(2)))
        at = [t * strides[1] + h * strides[2] for t, h in itertools.product(range(T), range(H))]
        at.sort()
        want = any(b - a < 128 for a, b in zip(at, at[1:]))
        assert refused(lib, 0, T, H, strides) == want, (T, H, strides)
        seen[want] += 1
    assert min(seen.values()) > 500

"""The limit of the latent kernels' waits, without a GPU."""
import threading

import pytest

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

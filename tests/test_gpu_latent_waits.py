"""The waits within the latent kernels run out in bounded time, report it and leave the GPU usable: with
stalled waits a kernel's first copy is announced and never made, so that the roles that wait for it,
and those that wait for them, give up."""
import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import latent_models as lm
from tests.test_gpu_latents import gen, normal, prompts, status_word
from tests.test_gpu_timeout import LIMIT_NS, gpu_ms

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


@pytest.fixture
def stalled():
    """Calls `fn` with waits of 1 ms that run out; ms on the GPU."""
    def call(fn):
        hs.set_latent_waits(LIMIT_NS, stall=True)
        try:
            return gpu_ms(fn)
        finally:
            hs.set_latent_waits()
    yield call
    hs.set_latent_waits()


def in_time(ms):
    assert 0.5 <= ms <= 50.0, f"a stalled call took {ms:.3f} ms on the GPU with a 1 ms limit of a wait"


def test_prompts(stalled):
    lens, H = [(200, 300), (1, 128), (140, 90)], 3
    q, k, r, v, qs, ks = prompts(lens, H, BF16, 5)
    o, lse = torch.full((341, H, 128), 7.0, dtype=BF16, device="cuda"), torch.full((341, H), 7.0, device="cuda")
    word = status_word()

    def call():
        hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, status=word)

    in_time(stalled(call))
    assert int(word) == hs.HS_STATUS_TIMEOUT
    assert (torch.isnan(o) | (o == 7)).all() and (torch.isnan(lse) | (lse == 7)).all()
    assert torch.isnan(o[:200]).any()
    word.zero_()
    call()
    assert int(word) == 0
    a, c = 0, 0
    for lq, lk in lens:
        wo, wl, bo, bl = lm.attend(q[a:a + lq], k[c:c + lk], r[c:c + lk], v[c:c + lk], 0.1, True, BF16)
        assert lm.near(o[a:a + lq], wo, bo) and lm.near(lse[a:a + lq], wl, bl)
        a, c = a + lq, c + lk

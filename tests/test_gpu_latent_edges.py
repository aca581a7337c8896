"""The latent operators where prompts' bounds, values or sizes are unusual, against the 64-bit models."""
import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import latent_models as lm
from tests.test_gpu_latents import gen, normal, prompts, status_word

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


def starts(*at):
    return torch.tensor(at, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ bounds
@pytest.mark.parametrize("before,behind", [(0, 0), (30, 0), (31, 5), (67, 40)])
def test_a_prompt_behind_descending_starts_does_not_cost_another_its_rows(before, behind):
    """Starts that descend and rise again: the rows stay the first prompt's that has them, and the prompts
    behind, of which none is left out, get theirs."""
    H, rows = 2, 1256
    q, k, r, v, *_ = prompts([(rows, rows + 700)], H, BF16, 3)
    head = [0] * before  # prompts without rows
    qs = starts(*head, 0, 1000, 0, 1000, 1256, *([1256] * behind))
    lens = [0] * before + [900, 5, 300, 400] + [0] * behind
    ks = starts(0, *torch.tensor(lens).cumsum(0).tolist())
    o, lse = torch.full((rows, H, 128), 7.0, dtype=BF16, device="cuda"), torch.full((rows, H), 7.0, device="cuda")
    word = status_word()
    hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, status=word)
    assert int(word) == hs.HS_STATUS_RANGE
    for a, b, c, d in ((0, 1000, 0, 900), (1000, 1256, 1205, 1605)):
        wo, wl, bo, bl = lm.attend(q[a:b], k[c:d], r[c:d], v[c:d], 0.1, True, BF16)
        assert lm.near(o[a:b], wo, bo) and lm.near(lse[a:b], wl, bl), (a, b)


@pytest.mark.parametrize("rows,keys", [(0, 20), (0, 0), (5, 0)])
def test_starts_outside_tensors_without_rows_or_keys_are_reported(rows, keys):
    H = 3
    q, k, r, v, *_ = prompts([(rows, keys)], H, BF16, 3)
    o, lse = torch.full((rows, H, 128), 7.0, dtype=BF16, device="cuda"), torch.full((rows, H), 7.0, device="cuda")
    for qs, ks, bad in ((starts(0, rows), starts(0, keys), False), (starts(0, rows + 1), starts(0, keys), True),
                        (starts(0, 0, rows, rows), starts(0, 0, keys, keys + 1), True), (starts(*[0] * 50, -1), starts(*[0] * 51), True)):
        word = status_word()
        hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, status=word)
        assert int(word) == (hs.HS_STATUS_RANGE if bad else 0)
        hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1)
        torch.cuda.synchronize()

"""Scores of the page attention where their evaluation can lose them -- caps of every size,
biases that grow with the distance, keys that are NaN or -inf before any other is seen --
against the definition in 64 bits, with bounds relative to the scores themselves."""
import math

import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import page_models as pm
from tests.test_gpu_pages import case, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


def tight(c, scale, cap=0.0, slopes=None):
    """o and lse of the last query token in 64 bits, and the bounds (o, lse, tol_o, tol_l), as in
    page_models.attend but for the two that matter here:
      * the cap's tanh is within 2^-20 of its own value: below .4 of the cap it is a polynomial
        off by 2^-22, above it 1 - 2 / (1 + e^2y), whose exponential (2^-22.5, weighted by at most
        .43), sum (2^-24, 1.4) and reciprocal (2^-23, 1.4) are off relative to at least .38;
      * a bias counts from the nearest key, or from the farthest where it grows with the distance.
    """
    T, H, D = c["shape"]
    B, Tq, Hq, _ = c["q"].shape
    G = Hq // H
    half_step = 2.0 ** -8 if c["q"].dtype is torch.bfloat16 else 2.0 ** -11
    o = torch.zeros((B, Hq, D), dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        ok = (c["slots"][b] >= 0) & (c["sel"][b] >= 0)
        k, v = (x.flatten(0, 1) for x in pm.read(c["pages"][b][c["slots"][b][ok].long()], c["shape"]))
        pos = (c["sel"][b][ok].long()[:, None] * T + torch.arange(T)).reshape(-1)
        here = int(c["lengths"][b]) - 1
        see = pos <= here
        k, v, p = k[see], v[see], pos[see]
        for h in range(H if p.numel() else 0):
            r = slice(h * G, (h + 1) * G)
            q = c["q"][b, -1, r].double()
            x = q @ k[:, h].T * scale
            eps = D * 2.0 ** -23 * abs(scale) * (q.abs() @ k[:, h].abs().T)
            if cap:
                x = cap * torch.tanh(x / cap)
                eps = eps + 2.0 ** -20 * x.abs()
            eps = eps + 2.0 ** -21 * x.abs()
            lost = 0.0
            if slopes is not None:
                sl = slopes[r].double()[:, None]
                x = x - sl * (here - p).double()
                far = torch.where(sl < 0, p - p.min(), p.max() - p).double()
                eps = eps + 2.0 ** -21 * sl.abs() * far
                lost = 2.0 ** -21 * sl[:, 0].abs() * torch.where(sl[:, 0] < 0, here - p.min(), here - p.max()).double()
            total = torch.logsumexp(x, -1)
            w = torch.exp(x - total[:, None])
            out = w @ v[:, h]
            mag = v[:, h].abs()
            moved = (w * (eps + 2.0 ** -20)).sum(-1, keepdim=True)
            tol = (w * (eps + 2.0 ** -20 + 2.0 ** -11 + (p.numel() / 16 + 20) * 2.0 ** -23)) @ mag + moved * out.abs()
            o[b, r], lse[b, r] = out, total
            tol_o[b, r] = 1.05 * (tol + 2.0 ** -25 * mag.sum(0) + half_step * out.abs() + 2.0 ** -25)
            tol_l[b, r] = 1.05 * (moved[:, 0] + 2.0 ** -21 * (total.abs() + 1) + lost)
    return o, lse, tol_o, tol_l


def check(c, scale, cap=0.0, slopes=None):
    mods = {"softcap": cap} if slopes is None else {"softcap": cap, "slopes": slopes}
    o, lse = run(c, scale, **mods)
    ro, rl, to, tl = tight(c, scale, cap, slopes)
    off_o, off_l = ((o[:, -1] - ro).abs() / to).max(), ((lse[:, -1] - rl).abs() / tl).max()
    assert off_o <= 1 and off_l <= 1, f"o off by {off_o:.3g} of its bound, lse by {off_l:.3g}"


CAPS = [1e-3, 1.0, 50.0, 1e3, 1e6, 1e12, 1e29]


@pytest.mark.parametrize("cap", CAPS)
def test_a_capped_score_is_right_relative_to_itself(cap):
    """One key a request, whose lse is its score: from 2^-24 of the cap to 16 times it."""
    g = torch.Generator().manual_seed(1)
    j = torch.arange(-24, 5).repeat_interleave(16)
    x = cap * 2.0 ** j * (1 + torch.rand(j.numel(), generator=g))
    x = torch.where(torch.rand(j.numel(), generator=g) < 0.5, -x, x).to(torch.bfloat16)
    B = x.numel()
    page = torch.zeros(16 * 64 * 9 // 8, dtype=torch.uint8)
    page[0], page[16 * 32] = 2, 0x78  # token 0: 1 in dimension 0, the scale of one
    q = torch.zeros((B, 1, 1, 64), dtype=torch.bfloat16)
    q[:, 0, 0, 0] = x
    zero = torch.zeros((B, 1), dtype=torch.int32)
    c = dict(shape=(16, 1, 64), q=q, pages=page.expand(B, 1, -1).contiguous(), slots=zero, sel=zero,
             lengths=torch.ones(B, dtype=torch.int32))
    _, lse = run(c, 1.0, softcap=cap)
    want = cap * torch.tanh(x.double() / cap)
    # the tanh 2^-20; the score, its scale and the cap in log2 units and back: 2^-21; the
    # logarithm of the sum, one, 2^-22
    off = (lse[:, 0, 0] - want).abs() / (1.5 * 2.0 ** -20 * want.abs() + 2.0 ** -22)
    assert off.max() <= 1, f"off by {off.max():.3g} of the bound at {float(x[off.argmax()]):.4g}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cap", CAPS)
def test_attention_with_caps_of_every_size(cap, dtype):
    c = case(2, 2, 3, 128, 16, 9, 12, [144, 100], dtype=dtype, seed=11, qsize=3.0)
    check(c, 128 ** -0.5, cap)
    c = case(2, 1, 16, 64, 32, 6, 6, [192, 33], dtype=dtype, seed=12)
    check(c, 0.125, cap, 2.0 ** -torch.arange(1.0, 17.0))
    check(case(1, 2, 5, 256, 16, 40, 40, [640], dtype=dtype, seed=13), 0.0625, cap)


@pytest.mark.parametrize("mods", [{}, {"softcap": 8.0}, {"slopes": 2.0 ** -torch.arange(1.0, 17.0)}])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_key_that_no_other_key_precedes(D, mods):
    """The first key of each sequence is NaN for one head: its rows see nothing else at length 1,
    and at length 3 the others. Such rows are NaN, not rows without a key."""
    c = case(4, 2, 8, D, 16, 1, 1, [1, 3, 1, 2], seed=D)
    want, wl = run(c, 0.1, **mods)
    _, scale_at = pm.offsets((16, 2, D))
    for b in range(3):  # the fourth has none
        c["pages"][b, c["slots"][b, 0], scale_at[0, 0, 0, 0]] = 0xFF
    o, lse = run(c, 0.1, **mods)
    assert torch.isnan(o[:3, 0, :8]).all() and torch.isnan(lse[:3, 0, :8]).all()
    assert torch.equal(o[:, 0, 8:], want[:, 0, 8:]) and torch.equal(lse[:, 0, 8:], wl[:, 0, 8:])
    assert torch.equal(o[3], want[3]) and torch.equal(lse[3], wl[3])


def minus_infinity(lens, k, last):
    """Requests whose scores are -inf in f32 (-3e38 x 4 x 100) at positions below `last`, 0 from it."""
    c = case(len(lens), 1, 8, 64, 16, k, k, lens, seed=5)
    c["q"].zero_()
    c["q"][..., 0] = -3e38
    code_at, scale_at = pm.offsets((16, 1, 64))
    for b in range(len(lens)):
        for j in range(k):
            if c["sel"][b, j] >= 0:
                p = int(c["sel"][b, j]) * 16 + torch.arange(16)
                page = c["pages"][b, c["slots"][b, j]]
                page[code_at[0, :, 0, 0]] = torch.where(p < last, 6, 0).to(torch.uint8)  # 4 and, beside it, 0
                page[scale_at[0, :, 0, 0]] = 0x78
    return c


def test_scores_of_minus_infinity_are_not_seen():
    """Before any other key is seen, next to masked ones: no NaN, and no part in the result."""
    slopes = 2.0 ** -torch.arange(8.0, 16.0)
    c = minus_infinity([1, 9, 40], 4, 1000)
    for mods in ({}, {"slopes": slopes}):
        o, lse = run(c, 100.0, **mods)
        assert not o.any() and torch.isneginf(lse).all()
    c = minus_infinity([960, 955], 60, 480)
    mods = dict(slopes=slopes, start=torch.tensor([320, 330]), prefix=torch.tensor([8, 5]))
    mods = {n: x.int() if n != "slopes" else x for n, x in mods.items()}
    o, lse = run(c, 100.0, **mods)
    ro, rl, to, tl = pm.attend(c["shape"], c["q"], c["pages"], c["slots"], c["sel"], c["lengths"], 100.0, **mods)
    assert ((o - ro).abs() <= to).all() and ((lse - rl).abs() <= tl).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G,D", [(2, 4, 64), (1, 8, 128), (1, 12, 256), (1, 24, 64)])
def test_biases_that_grow_with_the_distance(H, G, D, dtype):
    """Slopes below zero over 1.6 million tokens, beside ones above: the far keys then carry the
    weight, and their biases' differences decide."""
    c = case(2, H, G, D, 16, 64, 64, [1600000, 1400007], dtype=dtype, seed=9)
    near = (c["sel"] >= 0) & (torch.arange(64) % 4 != 0)
    c["sel"] = torch.where(near, c["sel"] % 40 + 17, c["sel"])  # several pages share the far end
    slopes = 2.0 ** -(torch.arange(H * G) % 8).float() * torch.where(torch.arange(H * G) % 3 == 0, 1.0, -1.0)
    check(c, D ** -0.5, 0.0, slopes)
    check(c, D ** -0.5, 20.0, slopes)

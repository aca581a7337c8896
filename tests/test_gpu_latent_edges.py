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


# ------------------------------------------------------------------------ weights
def small_weights(n, less, dtype):
    """A prompt of one row: key n weighs 1, and each of the n before it 2^-less; dimension 0 of the
    values is theirs alone, dimension 1 the dominant key's, dimension 2 everyone's."""
    q, k, r, v, qs, ks = prompts([(1, n + 1)], 1, dtype, 12)
    for t in (q, k, r, v):
        t.zero_()
    q[0, 0, 0], k[n, 0, 0] = 1, less * 0.6931471805599453
    v[:n, 0, 0], v[n, 0, 1], v[:, 0, 2] = 1, 1, 1
    return q, k, r, v, qs, ks


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,less,first", [(16383, 25.5, True), (16383, 25.5, False), (4000, 23.3, True), (100000, 27.0, True), (100000, 27.0, False)])
def test_weights_far_below_the_largest_are_not_lost(n, less, first, dtype):
    """Many keys of weights that half precision holds poorly or not at all, behind a dominant key (whose
    maximum is then there from the first tile) or ahead of it.

    A weight w is rounded to the operands' type: by half a step u of itself, and in half precision by 2^-25
    at the least; weights being held at 2^7 times their size or more, that is 2^-32 of the largest. exp2,
    the score's and the exponent's f32 roundings, 2^-24 of at most 18 each, change it by 2^-18 of itself at
    most; sums of n terms by n 2^-23; the result is rounded, by 2^-25 at the least."""
    q, k, r, v, qs, ks = small_weights(n, less, dtype)
    if first:
        for t in (k, v):
            t.copy_(t.flip(0))
    o, lse = torch.full((1, 1, 128), 7.0, dtype=dtype, device="cuda"), torch.full((1, 1), 7.0, device="cuda")
    word = status_word()
    hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 1.0, causal=False, status=word)
    assert int(word) == 0
    w = torch.softmax(k[:, 0, 0].double(), 0)
    want, u = torch.einsum("k,kd->d", w, v[:, 0].double()), lm.half_step(dtype)
    least = 2.0 ** -25 if dtype == F16 else 2.0 ** -134
    bound = (2 * u + 2.0 ** -18 + (n + 16) * 2.0 ** -23) * want + 2.0 ** -32 * v[:, 0].double().sum(0) + least
    assert (want[0] > 2.0 ** -13) and ((o[0, 0].double() - want).abs() <= bound).all(), (o[0, 0, :3], want[:3], bound[:3])
    ref = torch.logsumexp(k[:, 0, 0].double(), 0)
    assert abs(float(lse) - float(ref)) <= 2.0 ** -18 + (n + 16) * 2.0 ** -23 + 2.0 ** -22 * float(ref)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale", [0.5, 5.0])
def test_maxima_that_grow_in_small_steps(scale, dtype):
    """The kept maximum lags behind by up to 2^8: weights above 1, which half precision has to hold too."""
    n = 2000
    q, k, r, v, qs, ks = prompts([(130, n)], 2, dtype, 14)
    q.abs_()
    k.copy_((torch.arange(n, device="cuda")[:, None, None] / 2048.0 * torch.ones_like(k)).to(dtype))
    o, lse = torch.empty((130, 2, 128), dtype=dtype, device="cuda"), torch.empty((130, 2), device="cuda")
    hs.attend_prompts(q, k, r, v, qs, ks, o, lse, scale, causal=False)
    wo, wl, bo, bl = lm.attend(q, k, r, v, scale, False, dtype)
    assert lm.near(o, wo, bo) and lm.near(lse, wl, bl)


# ------------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lq,lk", [(256, 306), (256, 256), (300, 300), (130, 1000), (256, 100), (40, 41), (600, 615)])
def test_what_an_infinite_value_reaches_under_a_causal_mask(lq, lk, dtype):
    """Rows that see the key: what the definition gives. Rows that do not: nothing, unless one of the same
    128 rows sees the key or one of the 15 before it (then the row may be NaN)."""
    H, scale = 2, 0.1
    q, k, r, v, qs, ks = prompts([(lq, lk)], H, dtype, 13)
    tiles = [(a, min(a + 128, lq)) for a in range(0, lq, 128)]
    seen = [max(0, min(lk, b + lk - lq)) for _, b in tiles]  # by a tile's last row, which sees the most
    keys = {x for s in seen for x in (s - 1, s, -(-s // 16) * 16 - 1, -(-s // 16) * 16, s + 40) if 0 <= x < lk}
    for key in sorted(keys):
        vv = v.clone()
        vv[key, 0, 5], vv[key, 1, 6] = float("inf"), float("nan")
        o, lse = torch.full((lq, H, 128), 7.0, dtype=dtype, device="cuda"), torch.full((lq, H), 7.0, device="cuda")
        word = status_word()
        hs.attend_prompts(q, k, r, vv, qs, ks, o, lse, scale, status=word)
        assert int(word) == 0
        wo, wl, bo, bl = lm.attend(q, k, r, vv, scale, True, dtype)
        assert lm.near(lse, wl, bl)
        for (a, b), s in zip(tiles, seen):
            row = torch.arange(a, b, device="cuda")
            free = (key > row + lk - lq) & (key < -(-s // 16) * 16)  # not seen, but within the products
            for h, d in ((0, 5), (1, 6)):
                assert (torch.isnan(o[a:b, h, d]) | ~free | (wo[a:b, h, d] == 0)).all()
                o[a:b, h, d] = torch.where(free, wo[a:b, h, d].to(dtype), o[a:b, h, d])
        assert lm.near(o, wo, bo), (key, seen)


# ------------------------------------------------------------------------ entries
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_magnitude_reads_back_as_its_code_times_the_scale(dtype):
    """Each number of the type as the largest of a block, beside fractions of it, in both output types:
    the 64-bit product rounded once, infinite where that is too large (2^128 in bf16)."""
    a = torch.arange(0, 32768, dtype=torch.int16).view(dtype).cuda()
    a = a[torch.isfinite(a)]
    a = a[:a.numel() // 4 * 4]
    x = (a.double()[:, None] * torch.linspace(1, -1, 128, device="cuda", dtype=torch.float64)).to(dtype)
    latent = x.view(-1, 512)
    n = latent.shape[0]
    entries, rope = torch.zeros((n, 656), dtype=torch.uint8, device="cuda"), torch.zeros((n, 64), dtype=dtype, device="cuda")
    hs.write_latents(latent, rope, torch.arange(n, device="cuda"), entries)
    want, _ = lm.values(entries)
    # half a step of an E4M3 code, or of its smallest ones
    assert ((want - latent.double()).abs() <= torch.maximum(2.0 ** -4 * latent.double().abs(), 2.0 ** -10 * lm.scales(latent).repeat_interleave(128, 1))).all()
    assert (want.abs().amax() == 2.0 ** 128) == (dtype == BF16)
    for out in (BF16, F16):
        lo, ro = torch.empty((1, n, 512), dtype=out, device="cuda"), torch.empty((1, n, 64), dtype=out, device="cuda")
        hs.read_latents(entries.view(1, n, 656), torch.arange(n, dtype=torch.int32, device="cuda").view(1, n), lo, ro)
        got, most = lo[0].double(), torch.finfo(out).max
        step = 2.0 ** -133 if out == BF16 else 2.0 ** -24  # the smallest number
        large = want.abs() >= most * (1 + lm.half_step(out) / 2)
        assert torch.isinf(got[large]).all() and torch.equal(torch.sign(got[large]), torch.sign(want[large]))
        exact = want[~large] if out == BF16 else want[~large].to(torch.float32).to(out).double()
        assert ((got[~large] - exact).abs() <= (step / 2 if out == BF16 else 0)).all()


# ------------------------------------------------------------------------ outputs
@pytest.mark.parametrize("n,H", [(1, 114), (1, 115), (16, 114), (17, 57), (17, 58), (1, 153), (33, 160), (65, 100), (95, 101), (300, 31), (1100, 3)])
def test_outputs_at_sizes_about_the_kernels_limits(n, H):
    g = gen(n + H)
    x = (normal(g, n, H, 520) * torch.exp(2 * normal(g, n, H, 1)))[..., 4:516]
    up = (normal(g, H, 130, 512) * 512 ** -0.5).to(BF16)[:, 1:129]
    back = torch.full((n + 33, H, 128), 7.0, dtype=BF16, device="cuda")
    word = status_word()
    hs.expand_outputs(x, up, back[:n], status=word)
    ref = torch.einsum("nhc,hec->nhe", x.double(), up.double())
    size = torch.einsum("nhc,hec->nhe", x.double().abs(), up.double().abs())
    # x's rounding and the result's, and f32 sums of 512
    assert ((back[:n].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 514 * 2.0 ** -23) * size).all()
    assert int(word) == 0 and (back[n:] == 7).all()


@pytest.mark.parametrize("n,H", [(1, 2), (1, 128), (16, 5), (40, 20), (65, 2), (70, 128), (300, 9), (1000, 30)])
def test_outputs_take_sums_of_latents_as_they_are(n, H):
    """Sums that differ by less than a step of bf16, which the matrices make all of the result: f32 rows are taken
    to within 2^-15, with f32 sums of 1024 products, and the result is rounded."""
    x = 1 + torch.randint(-5, 6, (n, H, 512), generator=gen(n), device="cuda") * 2.0 ** -10
    up = torch.randint(0, 2, (H, 128, 512), generator=gen(H), device="cuda").to(BF16) * 2 - 1
    up[..., 1::2] = -up[..., ::2]  # pairs of opposite signs
    out = torch.empty((n, H, 128), dtype=BF16, device="cuda")
    hs.expand_outputs(x, up, out)
    want = torch.einsum("nhc,hec->nhe", x.double(), up.double())
    size = torch.einsum("nhc,hec->nhe", x.double().abs(), up.double().abs())
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -15 + 1026 * 2.0 ** -23) * size).all()


@pytest.mark.parametrize("n,H", [(3, 2), (200, 40)])
def test_outputs_of_rows_that_are_not_finite(n, H):
    """Infinities stay infinite, through the largest numbers too, and NaNs NaNs, whatever their bits."""
    x, up = normal(gen(1), n, H, 512), normal(gen(2), H, 128, 512).to(BF16).abs() + 1
    x[0, 0, 5], x[1, 0, 6], x[2, 0, 7] = float("inf"), float("-inf"), float("nan")
    x[1, 1] = 0
    x[1, 1, 9] = torch.finfo(torch.float32).max
    x.view(torch.int32)[2, 1, 511] = 0x7F800001
    out = torch.empty((n, H, 128), dtype=BF16, device="cuda")
    hs.expand_outputs(x, up, out)
    assert (out[0, 0] == float("inf")).all() and (out[1, 0] == float("-inf")).all()
    assert torch.isnan(out[2, 0]).all() and torch.isnan(out[2, 1]).all()
    assert (out[1, 1] == float("inf")).all()  # times 1 or more: too large, but for 1 itself, which rounds up in bf16
    assert torch.isfinite(out[0, 1]).all()
    if n > 3:
        assert torch.isfinite(out[3:]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_the_lse_of_a_single_key_is_its_score(dtype):
    """Whole numbers, whose products and sums are exact: the score's factor (of two roundings, 2^-24 each), its
    product, the sum with the weights' logarithm and the way back are off by 5 2^-24, the logarithm of a sum
    of about 1 by 2^-22."""
    n, H = 300, 3
    q, k, r, v, *_ = prompts([(n, n)], H, dtype, 17)
    for t in (q, k, r):
        t.copy_(torch.randint(-4, 5, t.shape, generator=gen(t.numel()), device="cuda"))
    at = torch.arange(n + 1, dtype=torch.int32, device="cuda")  # n prompts of a row and a key
    o, lse = torch.empty((n, H, 128), dtype=dtype, device="cuda"), torch.empty((n, H), device="cuda")
    hs.attend_prompts(q, k, r, v, at, at, o, lse, 0.0625)
    kk = torch.cat((k, r[:, None].expand(-1, H, -1)), -1)
    want = (q.double() * kk.double()).sum(-1) * 0.0625
    assert torch.equal(o, v)
    assert ((lse.double() - want).abs() <= 5 * 2.0 ** -24 * want.abs() + 2.0 ** -22).all()

"""4-bit pages on the GPU against the 64-bit model of tests/page_models.py: written bytes and
read values are equal, the attention is within the bound that page_models.attend derives."""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
import tracegen
from tests import page_models as pm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ writing and reading
def tokens(n, H, D, dtype, seed):
    """Rows of very different sizes, with exact ties, zeros and signed zeros among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, H, D), generator=g) * torch.exp(3 * torch.randn((n, H, D // 16, 1), generator=g)).expand(
        n, H, D // 16, 16).reshape(n, H, D)
    ties = torch.randint(-48, 49, (n, H, D), generator=g) / 8.0
    x = torch.where(torch.rand((n, H, 1), generator=g) < 0.4, ties, x)
    x[torch.rand((n, H, D), generator=g) < 0.05] = -0.0
    return x.to(dtype)


@pytest.mark.parametrize("shape,n,dtype", [
    ((16, 8, 128), 64, torch.bfloat16), ((16, 1, 64), 1, torch.float16), ((32, 3, 64), 37, torch.bfloat16),
    ((48, 2, 256), 29, torch.float16), ((256, 5, 128), 300, torch.bfloat16), ((16, 2, 128), 0, torch.bfloat16)])
def test_written_bytes_and_read_values(shape, n, dtype):
    T, H, D = shape
    P = n // T + 3
    ref = pm.random_pages(P, shape, n)
    pages = ref.cuda()
    k, v = tokens(n, H, D, dtype, 1), tokens(n, H, D, dtype, 2)
    dest = torch.randperm(P * T, generator=torch.Generator().manual_seed(n))[:n]
    dest[3::7] = -1 - dest[3::7]  # padding
    word = status_word()
    hs.write_tokens(shape, k.cuda(), v.cuda(), dest.cuda(), pages, status=word)
    pm.write(ref, shape, k, v, dest)
    assert torch.equal(pages.cpu(), ref)
    slots = torch.randperm(P)[: P - 1].to(torch.int32)
    slots[0] = -1
    ko = torch.full((1, (P - 1) * T, H, D), 7.0, dtype=dtype, device="cuda")
    vo = ko.clone()
    hs.read_pages(shape, pages.view(1, P, -1), slots.cuda().view(1, -1), ko, vo, status=word)
    kr, vr = (x[slots.clamp(min=0).long()].flatten(0, 1)[None] for x in pm.read(ref, shape))
    kr[:, :T], vr[:, :T] = 0, 0
    assert torch.equal(ko.cpu().double(), kr) and torch.equal(vo.cpu().double(), vr)
    assert int(word) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_magnitude_as_a_blocks_largest(dtype):
    """Each positive number of the type (infinities and NaNs too) as the largest of a block,
    beside a half, a quarter and an odd fraction of it."""
    shape = (16, 4, 128)
    bits = torch.arange(1, 32768, dtype=torch.int16)
    a = bits.view(dtype)
    x = torch.zeros((32768, 16), dtype=dtype)
    x[1:, 0], x[1:, 3] = a, -(a.float() / 2).to(dtype)
    x[1:, 9], x[1:, 15] = (a.float() / 4).to(dtype), (a.float() * 0.2917).to(dtype)
    x = x.view(1024, 4, 128).contiguous()[:1023]
    ref = torch.zeros((64, 9216), dtype=torch.uint8)
    pages = ref.cuda()
    dest = torch.arange(1023)
    hs.write_tokens(shape, x.cuda(), x.flip(0).cuda(), dest.cuda(), pages)
    pm.write(ref, shape, x, x.flip(0), dest)
    assert torch.equal(pages.cpu(), ref)


def test_infinities_and_nans_make_nan_blocks():
    shape = (16, 1, 64)
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16)
    k[0, 0, 5], k[1, 0, 17], k[2, 0, 63] = math.inf, math.nan, -math.inf
    pages = torch.zeros((1, 1152), dtype=torch.uint8, device="cuda")
    hs.write_tokens(shape, k.cuda(), k.cuda(), torch.arange(3).cuda(), pages)
    out = torch.empty((1, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    hs.read_pages(shape, pages[None], torch.zeros((1, 1), dtype=torch.int32, device="cuda"), out, out.clone())
    bad = torch.isnan(out[0, :3, 0].cpu().float()).view(3, 4, 16)
    want = torch.zeros((3, 4, 16), dtype=torch.bool)
    want[0, 0], want[1, 1], want[2, 3] = True, True, True
    assert torch.equal(bad, want)
    # a block of ones: the scale nearest to 1/6 is 11/64, and 1 over it, 5.82, rounds to 6
    assert torch.equal(out[0, :3, 0].cpu().float().view(3, 4, 16)[~want], torch.full((9 * 16,), 6 * 11 / 64))


def test_strides_padding_range_and_pinned_pages():
    shape, n, P = (16, 3, 64), 20, 2
    qkv = tokens(n, 10, 64, torch.float16, 4).cuda()  # q, k and v of one projection
    k, v = qkv[:, 4:7], qkv[:, 7:10]
    dest = torch.arange(n) * 3 % 47
    dest[2], dest[9], dest[11] = 32, -1, 2**62  # past the pages, padding, far past
    ref = pm.random_pages(P, shape, 9)
    pages = ref.clone().pin_memory()
    word = status_word()
    hs.write_tokens(shape, k, v, dest.cuda(), pages, status=word)
    torch.cuda.synchronize()
    pm.write(ref, shape, k.cpu(), v.cpu(), dest)
    assert torch.equal(pages, ref)
    assert int(word) == hs.HS_STATUS_RANGE
    out = torch.empty((1, 32, 3, 64), dtype=torch.float16, device="cuda")
    word.zero_()
    hs.read_pages(shape, ref.cuda()[None], torch.tensor([[2, 1]], dtype=torch.int32, device="cuda"), out, out.clone(), status=word)
    assert int(word) == hs.HS_STATUS_RANGE and not out[:, :16].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_that_are_16_byte_but_not_32_byte_aligned(dtype):
    shape, n = (32, 2, 128), 37
    base = tokens(n, 3, 128, dtype, 6).reshape(-1).cuda()
    k = base[8:8 + n * 256].view(n, 2, 128)
    v = torch.as_strided(base, (n, 2, 128), (264, 128, 1), 16)  # token stride of 33 times 16 bytes
    assert k.data_ptr() % 32 == 16
    dest = torch.arange(n) + 5
    ref = pm.random_pages(2, shape, 3)
    pages = ref.cuda()
    hs.write_tokens(shape, k, v, dest.cuda(), pages)
    pm.write(ref, shape, k.cpu(), v.cpu(), dest)
    assert torch.equal(pages.cpu(), ref)
    out = torch.zeros(2, 64 * 256 + 16, dtype=dtype, device="cuda")
    ko, vo = (x[8:8 + 64 * 256].view(1, 64, 2, 128) for x in out)
    slots = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    hs.read_pages(shape, pages[None], slots, ko, vo)
    for got, want in zip((ko, vo), pm.read(ref, shape)):
        assert torch.equal(got.cpu().double()[0], want[[1, 0]].flatten(0, 1))
    assert not out[:, :8].any() and not out[:, -8:].any()
    odd = torch.zeros(n * 256 + 8, dtype=dtype, device="cuda")[4:4 + n * 256].view(n, 2, 128)
    with pytest.raises(hs.HsError, match="aligned"):
        hs.write_tokens(shape, odd, odd, dest.cuda(), pages)


def test_refuses_tensors_that_are_not_on_the_device():
    shape = (16, 1, 64)
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    pages = torch.zeros((1, 1152), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        hs.write_tokens(shape, k, k, torch.zeros(1, dtype=torch.int64, device="cuda"), pages)
    with pytest.raises(ValueError):
        hs.write_tokens(shape, k.cuda(), k.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), pages.cpu())
    slots = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        hs.attend_pages(shape, q, pages[None], slots, slots, slots[0].cpu(), q.clone(), torch.zeros((1, 1, 1), device="cuda"), 1.0)


# -------------------------------------------------------------------------------- attention
def case(B, H, G, D, T, k, S, lens, Tq=1, dtype=torch.bfloat16, seed=0, qsize=1.0):
    shape, Hq = (T, H, D), H * G
    g = torch.Generator().manual_seed(seed)
    pages = pm.random_pages(B * S, shape, seed).view(B, S, T * H * D * 9 // 8)
    sel = torch.full((B, k), -1, dtype=torch.int32)
    slots = torch.full((B, k), -1, dtype=torch.int32)
    for b in range(B):
        held = max(0, -(-lens[b] // T))
        at = torch.randperm(held, generator=g)[:k]
        if held and k:  # the last page is always selected
            at = torch.cat([at[at != held - 1][: max(0, min(k, held) - 1)], torch.tensor([held - 1])])[:k]
            at = at[torch.randperm(len(at), generator=g)]
        where = torch.randperm(k, generator=g)[: len(at)]  # padding in between
        sel[b, where] = at.to(torch.int32)
        slots[b, where] = torch.randperm(S, generator=g)[: len(at)].to(torch.int32)
    q = (qsize * torch.randn((B, Tq, Hq, D), generator=g)).to(dtype)
    return dict(shape=shape, q=q, pages=pages, slots=slots, sel=sel, lengths=torch.tensor(lens, dtype=torch.int32))


def run(c, scale, stream=None, status=None, **mods):
    o = torch.full_like(c["q"], 9.0, device="cuda")
    lse = torch.full(c["q"].shape[:3], 9.0, device="cuda")
    mods = {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in mods.items()}
    cu = [c[n].cuda() for n in ("q", "pages", "slots", "sel", "lengths")]
    torch.cuda.synchronize()
    hs.attend_pages(c["shape"], *cu, o, lse, scale, status=status, stream=stream, **mods)
    torch.cuda.synchronize()
    return o.cpu().double(), lse.cpu().double()


def check(c, scale, got=None, **mods):
    o, lse = run(c, scale, **mods) if got is None else got
    model = {"cap" if n == "softcap" else n: x for n, x in mods.items()}
    ro, rl, to, tl = pm.attend(c["shape"], c["q"], c["pages"], c["slots"], c["sel"], c["lengths"], scale, **model)
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert not o[empty].any()
    lost = torch.isnan(rl)  # rows whose query is not finite
    assert torch.equal(torch.isnan(lse), lost) and torch.equal(torch.isnan(o).any(-1), lost)
    off = (o - ro).abs()[~lost] / to[~lost].clamp(min=2.0 ** -60)
    assert (off <= 1).all(), f"o off by {off.max():.2f} of its bound"
    at = ~empty & ~lost
    assert ((lse - rl)[at].abs() <= tl[at]).all(), f"lse off by {((lse - rl)[at].abs() / tl[at]).max():.2f} of its bound"


SHAPES = [
    # B, H, G, D, T, k, S, lens, Tq
    (1, 1, 1, 64, 16, 1, 1, [1], 1),
    (2, 2, 3, 128, 16, 3, 5, [16, 33], 1),
    (3, 1, 8, 128, 32, 4, 4, [15, 128, 97], 1),
    (1, 8, 8, 128, 16, 128, 140, [40000], 1),      # shares of one selection in a cluster
    (2, 3, 9, 128, 16, 9, 12, [144, 139], 1),      # two tiles of eight rows, the second ragged
    (2, 2, 16, 64, 48, 5, 7, [240, 200], 1),
    (1, 2, 33, 128, 16, 6, 6, [90], 1),            # more rows than one CTA takes
    (2, 1, 24, 64, 16, 20, 20, [320, 311], 1),
    (2, 2, 5, 256, 16, 7, 9, [100, 112], 1),
    (1, 1, 40, 256, 32, 3, 3, [77], 1),
    (2, 2, 4, 128, 16, 6, 8, [90, 3], 4),          # drafted tokens, one sequence shorter than them
    (2, 1, 7, 256, 64, 2, 3, [100, 65], 3),
    (3, 2, 2, 64, 16, 10, 12, [155, 160, 150], 2),
    (2, 1, 4, 64, 256, 40, 40, [10000, 9999], 1),  # whole pages of many tiles
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,H,G,D,T,k,S,lens,Tq", SHAPES)
def test_attention_matches_the_model(B, H, G, D, T, k, S, lens, Tq, dtype):
    check(case(B, H, G, D, T, k, S, lens, Tq, dtype, seed=D + k), D ** -0.5)


@pytest.mark.parametrize("B,H,G,D,T,k,S,lens,Tq", SHAPES)
def test_attention_with_cap_bias_and_document_masks(B, H, G, D, T, k, S, lens, Tq):
    c = case(B, H, G, D, T, k, S, lens, Tq, seed=k + 1, qsize=3.0)
    slopes = 2.0 ** (-8.0 * torch.arange(1, H * G + 1) / (H * G))
    start = torch.tensor([n // 2 for n in lens], dtype=torch.int32)
    prefix = torch.tensor([n // 9 for n in lens], dtype=torch.int32)
    scale = D ** -0.5
    check(c, scale, softcap=20.0)
    check(c, scale, slopes=slopes)
    check(c, scale, start=start, prefix=prefix)
    check(c, scale, start=start)
    check(c, scale, softcap=5.0, slopes=-0.01 * slopes, start=start, prefix=prefix)


def test_every_length_around_the_tiles():
    lens = list(range(0, 50)) + [-3]
    for D in (64, 128, 256):
        check(case(len(lens), 1, 2, D, 16, 4, 4, lens, seed=D), 0.1)
        check(case(len(lens), 1, 2, D, 16, 4, 4, lens, Tq=3, seed=D + 1), 0.1)


def test_rows_and_selections_that_leave_nothing():
    c = case(4, 2, 3, 128, 16, 5, 6, [80, 0, 70, 5])
    c["slots"][0] = -1                      # nothing resident
    c["sel"][2] += 100                      # pages past the length
    check(c, 0.1)
    start = torch.tensor([0, 0, 0, 5], dtype=torch.int32)  # the document begins behind the last key
    check(c, 0.1, start=start, prefix=torch.zeros(4, dtype=torch.int32))
    c = case(2, 1, 1, 64, 16, 0, 3, [10, 20])
    o, lse = run(c, 1.0)
    assert not o.any() and torch.isneginf(lse).all()
    c = case(0, 1, 1, 64, 16, 2, 3, [])
    run(c, 1.0)


def test_slots_out_of_range_are_left_out_and_reported():
    c = case(2, 1, 4, 128, 16, 6, 8, [96, 96])
    c["slots"][1, 2] = 8
    c["slots"][0, 1] = 2**31 - 1
    word = status_word()
    check(c, 0.1, got=run(c, 0.1, status=word))
    assert int(word) == hs.HS_STATUS_RANGE


def test_a_page_selected_twice_counts_twice():
    c = case(1, 1, 2, 64, 16, 4, 4, [64])
    c["sel"][0, 1], c["slots"][0, 1] = c["sel"][0, 0], c["slots"][0, 0]
    check(c, 0.2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_masked_places_hold_does_not_matter(D):
    """NaN and infinite scales in every key no query sees: past the length, before the document."""
    lens, T = [21, 64, 90], 32
    c = case(3, 2, 4, D, T, 3, 4, lens, Tq=2, seed=D)
    start = torch.tensor([7, 40, 0], dtype=torch.int32)
    prefix = torch.tensor([3, 0, 0], dtype=torch.int32)
    want = run(c, 0.1, start=start, prefix=prefix)
    check(c, 0.1, got=want, start=start, prefix=prefix)
    _, scale_at = pm.offsets((T, 2, D))
    for b in range(3):
        for j in range(3):
            if c["slots"][b, j] < 0:
                continue
            p = int(c["sel"][b, j]) * T + torch.arange(T)
            hidden = (p >= lens[b]) | ((p < start[b]) & (p >= prefix[b]))
            at = scale_at[:, hidden].reshape(-1)
            c["pages"][b, c["slots"][b, j], at] = torch.where(torch.arange(at.numel()) % 3 == 0, 0xF8, 0xFF).to(torch.uint8)
    got = run(c, 0.1, start=start, prefix=prefix)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nans_reach_the_rows_that_see_them_and_no_others(D):
    """The third drafted token's values hold a NaN block: the rows before it are untouched."""
    c = case(1, 1, 2, D, 16, 2, 2, [21], Tq=3, seed=D)
    want, wl = run(c, 0.1)
    last = int((c["sel"][0] == 1).nonzero()[0])
    _, scale_at = pm.offsets((16, 1, D))
    blk = 1
    c["pages"][0, c["slots"][0, last], scale_at[1, 4, 0, 16 * blk]] = 0xFF  # position 20, V
    got, gl = run(c, 0.1)
    assert torch.equal(got[0, :2], want[0, :2]) and torch.equal(gl, wl)
    nan = torch.isnan(got[0, 2])
    assert nan[:, 16 * blk:16 * blk + 16].all() and int(nan.sum()) == 2 * 16
    assert torch.equal(got[0, 2][~nan], want[0, 2][~nan])
    c["pages"][0, c["slots"][0, last], scale_at[0, 4, 0, 0]] = 0xFF  # and its key
    got, gl = run(c, 0.1)
    assert torch.equal(got[0, :2], want[0, :2]) and torch.equal(gl[0, :2], wl[0, :2])
    assert torch.isnan(got[0, 2]).all() and torch.isnan(gl[0, 2]).all()


def test_nan_keys_are_kept_by_the_join():
    """A NaN key in one page of many: every row that sees it is NaN, whichever warp met it."""
    c = case(1, 2, 4, 128, 16, 64, 64, [1024])
    _, scale_at = pm.offsets((16, 2, 128))
    c["pages"][0, c["slots"][0, 17], scale_at[0, 3, 0, 0]] = 0xFF
    o, lse = run(c, 0.1)
    assert torch.isnan(o[0, 0, :4]).all() and torch.isnan(lse[0, 0, :4]).all()
    assert torch.isfinite(o[0, 0, 4:]).all()


@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, 1e30), (torch.bfloat16, 1e-30), (torch.float16, 2e4),
                                        (torch.float16, 1e-5), (torch.bfloat16, 300.0)])
def test_queries_of_every_size(dtype, size):
    c = case(2, 2, 5, 128, 16, 9, 9, [140, 99], dtype=dtype, qsize=size)
    c["q"][0, 0, 1] = 0
    check(c, 0.5 / size)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales_of_zero_and_below(scale):
    check(case(2, 2, 3, 64, 16, 5, 5, [70, 33]), scale)


def test_scores_far_apart_and_far_below_zero():
    c = case(2, 1, 8, 128, 16, 40, 40, [640, 611], qsize=60.0)
    check(c, 1.0)
    c["q"] = c["q"].abs() * -1
    check(c, 3.0)


def test_distance_bias_of_far_pages():
    """No selected page is near: the bias is large, its differences decide."""
    c = case(2, 2, 4, 64, 16, 64, 64, [1600000, 1600000])
    c["sel"] = torch.where(c["sel"] >= 0, c["sel"] % 5000, c["sel"])
    slopes = 2.0 ** -torch.arange(1.0, 9.0)
    check(c, 0.1, slopes=slopes)


@pytest.mark.parametrize("k,H,D", [(9000, 1, 64), (2500, 2, 128)])
def test_long_selections(k, H, D):
    """More tiles in a share than are listed at a time."""
    c = case(1, H, 2, D, 16, k, k + 5, [16 * k + 100], seed=3)
    check(c, D ** -0.5)
    check(c, D ** -0.5, start=torch.tensor([9 * k], dtype=torch.int32), prefix=torch.tensor([100], dtype=torch.int32))


@pytest.mark.parametrize("H,G,D,Tq,mods", [(8, 8, 128, 1, {}), (4, 2, 128, 1, {"softcap": 9.0}), (2, 16, 128, 1, {}),
                                           (8, 8, 128, 4, {}), (4, 6, 64, 1, {}), (2, 8, 64, 4, {"softcap": 9.0}),
                                           (4, 8, 256, 1, {}), (2, 12, 256, 1, {"softcap": 9.0})])
def test_every_number_of_requests(H, G, D, Tq, mods):
    """The same two requests over and over: shared, whole and mixed jobs, from a few to many an SM."""
    k = 67
    c = case(2, H, G, D, 16, k, k, [67 * 16 - 3, 41 * 16], Tq, seed=D + H)
    scale = D ** -0.5
    slopes = 2.0 ** -torch.arange(1.0, H * G + 1) if mods else None
    ro, rl, to, tl = pm.attend(c["shape"], c["q"], c["pages"], c["slots"], c["sel"], c["lengths"], scale, cap=9.0 if mods else 0.0, slopes=slopes)
    ro, rl, to, tl = (x.cuda() for x in (ro, rl, to, tl))
    for n in (2, 4, 8, 10, 14, 20, 24, 26, 40, 60, 78, 100, 140, 200):
        cu = [c[x].cuda().repeat(n // 2, *[1] * (c[x].dim() - 1)) for x in ("q", "pages", "slots", "sel", "lengths")]
        o, lse = torch.empty_like(cu[0]), torch.empty(cu[0].shape[:3], device="cuda")
        hs.attend_pages(c["shape"], *cu, o, lse, scale, slopes=slopes.cuda() if mods else None, **mods)
        o, lse = o.double().view(n // 2, *ro.shape), lse.double().view(n // 2, *rl.shape)
        assert ((o - ro).abs() <= to).all(), n
        assert ((lse - rl).abs() <= tl).all(), n


def test_buffer_beyond_four_gigabytes():
    shape, S = (256, 8, 256), 8000  # 589824 bytes a page, 4.7 GB
    E = hs.PageShape(*shape).bytes
    pages = torch.empty((1, S, E), dtype=torch.uint8, device="cuda")
    small = pm.random_pages(2, shape, 1)
    slots = torch.tensor([[S - 1, 7300]], dtype=torch.int32)
    pages[0, slots[0].long()] = small.cuda()
    q = torch.randn((1, 1, 8, 256)).to(torch.bfloat16)
    sel = torch.tensor([[0, 1]], dtype=torch.int32)
    lengths = torch.tensor([300], dtype=torch.int32)
    o, lse = torch.empty_like(q, device="cuda"), torch.empty((1, 1, 8), device="cuda")
    hs.attend_pages(shape, q.cuda(), pages, slots.cuda(), sel.cuda(), lengths.cuda(), o, lse, 0.1)
    ro, rl, to, tl = pm.attend(shape, q, small[None], torch.tensor([[0, 1]]), sel, lengths, 0.1)
    assert ((o.cpu().double() - ro).abs() <= to).all() and ((lse.cpu().double() - rl).abs() <= tl).all()
    # a token written behind the fourth gigabyte, and its page read back
    k = tokens(1, 8, 256, torch.bfloat16, 5)
    pm.write(small, shape, k, k, torch.tensor([70]))
    hs.write_tokens(shape, k.cuda(), k.cuda(), torch.tensor([(S - 1) * 256 + 70], device="cuda"), pages[0])
    assert torch.equal(pages[0, S - 1].cpu(), small[0])
    out = torch.empty((1, 256, 8, 256), dtype=torch.bfloat16, device="cuda")
    hs.read_pages(shape, pages, slots[:, :1].contiguous().cuda(), out, out.clone())
    assert torch.equal(out.cpu().double()[0], pm.read(small[:1], shape)[0][0])


def test_strided_queries_and_outputs():
    c = case(3, 2, 4, 128, 16, 6, 6, [96, 90, 7], Tq=2)
    qkv = torch.zeros((3, 2, 12, 128), dtype=torch.bfloat16, device="cuda")
    qkv[:, :, :8] = c["q"].cuda()
    o = torch.full((8, 3, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 2, 8), device="cuda")
    hs.attend_pages(c["shape"], qkv[:, :, :8], *(c[n].cuda() for n in ("pages", "slots", "sel", "lengths")),
                    o.permute(1, 2, 0, 3), lse, 0.1)
    torch.cuda.synchronize()
    check(c, 0.1, got=(o.permute(1, 2, 0, 3).cpu().double(), lse.cpu().double()))


def test_another_stream_and_a_captured_graph():
    c = case(4, 2, 8, 128, 16, 40, 44, [640, 600, 17, 300])
    side = torch.cuda.Stream()
    check(c, 0.1, got=run(c, 0.1, stream=side))
    cu = [c[n].cuda() for n in ("q", "pages", "slots", "sel", "lengths")]
    o, lse = torch.zeros_like(cu[0]), torch.zeros(c["q"].shape[:3], device="cuda")
    k = tokens(4, 2, 128, torch.bfloat16, 3)
    kd, dest = k.cuda(), torch.full((4,), -1, dtype=torch.int64, device="cuda")
    ko = torch.empty((4, 640, 2, 128), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.write_tokens(c["shape"], kd, kd, dest, cu[1].view(4 * 44, -1))
        hs.attend_pages(c["shape"], *cu, o, lse, 0.1)
        hs.read_pages(c["shape"], cu[1], cu[2], ko, vo)
    for step in range(2):  # replays see new inputs
        if step:
            c["q"] = c["q"].flip(2).contiguous()
            cu[0].copy_(c["q"])
            new = torch.tensor([int(c["slots"][b, (c["sel"][b] == 0).nonzero()[0, 0]]) * 16 + b + b * 44 * 16
                                if (c["sel"][b] == 0).any() else -1 for b in range(4)])
            dest.copy_(new)
            pm.write(c["pages"].view(4 * 44, -1), c["shape"], k, k, new)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(c, 0.1, got=(o.cpu().double(), lse.cpu().double()))
        kr = pm.read(c["pages"].view(4 * 44, -1), c["shape"])[0].view(4, 44, 16, 2, 128)
        live = (c["slots"] >= 0)[:, :, None, None, None]
        want = torch.where(live, kr[torch.arange(4)[:, None], c["slots"].clamp(min=0).long()], 0.0).reshape(4, 640, 2, 128)
        assert torch.equal(ko.cpu().double(), want)


def test_dimensions_of_one_may_have_any_stride():
    c = case(1, 1, 4, 64, 16, 3, 3, [40])
    q = torch.as_strided(c["q"].cuda(), (1, 1, 4, 64), (3, 5, 64, 1))
    o, lse = torch.empty(4 * 64, dtype=q.dtype, device="cuda"), torch.empty((1, 1, 4), device="cuda")
    hs.attend_pages(c["shape"], q, *(c[n].cuda() for n in ("pages", "slots", "sel", "lengths")),
                    torch.as_strided(o, (1, 1, 4, 64), (1, 7, 64, 1)), lse, 0.1)
    check(c, 0.1, got=(o.view(1, 1, 4, 64).cpu().double(), lse.cpu().double()))
    k = torch.as_strided(tokens(1, 1, 64, torch.bfloat16, 1).cuda(), (1, 1, 64), (1, 2, 1))
    ref = torch.zeros((1, 1152), dtype=torch.uint8)
    pages = ref.cuda()
    hs.write_tokens((16, 1, 64), k, k, torch.tensor([3], device="cuda"), pages)
    pm.write(ref, (16, 1, 64), k.cpu(), k.cpu(), torch.tensor([3]))
    assert torch.equal(pages.cpu(), ref)


def test_rows_broadcast_over_tokens_and_heads():
    k = tokens(1, 1, 128, torch.float16, 2)
    ref = torch.zeros((2, 16 * 3 * 128 * 9 // 8), dtype=torch.uint8)
    pages = ref.cuda()
    dest = torch.tensor([4, 9, 31])
    hs.write_tokens((16, 3, 128), k.cuda().expand(3, 3, 128), k.cuda().expand(3, 3, 128), dest.cuda(), pages)
    pm.write(ref, (16, 3, 128), k.expand(3, 3, 128), k.expand(3, 3, 128), dest)
    assert torch.equal(pages.cpu(), ref)


def test_captured_between_a_fork_and_a_join():
    """Work of another stream, a copy and a fill directly before and after the calls of a graph."""
    c = case(3, 2, 8, 128, 16, 24, 30, [380, 17, 300])
    cu = [c[n].cuda() for n in ("q", "pages", "slots", "sel", "lengths")]
    o, lse = torch.zeros_like(cu[0]), torch.zeros(c["q"].shape[:3], device="cuda")
    q0, lens0, far, copy = torch.zeros_like(cu[0]), torch.zeros_like(cu[4]), torch.zeros_like(o), torch.zeros_like(o)
    hs.attend_pages(c["shape"], *cu, o, lse, 0.1)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            lens0.copy_(cu[4])
            hs.attend_pages(c["shape"], cu[0], *cu[1:4], lens0, far, torch.empty_like(lse), 0.1)
        q0.copy_(cu[0])
        main.wait_stream(side)
        hs.attend_pages(c["shape"], q0, *cu[1:4], lens0, o, lse, 0.1)
        hs.attend_pages(c["shape"], q0, *cu[1:4], lens0, o, lse, 0.1)
        copy.copy_(o)
    for _ in range(3):
        for x in (o, lse, q0, lens0, far, copy):
            x.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for x in (o, far, copy):
        check(c, 0.1, got=(x.cpu().double(), lse.cpu().double()))


def test_two_calls_at_once_on_two_streams():
    a, b = case(2, 8, 8, 128, 16, 128, 128, [30000, 2000], seed=1), case(2, 8, 8, 128, 16, 128, 128, [500, 2000], seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for c in (a, b):
        cu = [c[n].cuda() for n in ("q", "pages", "slots", "sel", "lengths")]
        outs.append((cu, torch.empty_like(cu[0]), torch.empty(c["q"].shape[:3], device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, (cu, o, lse), s in zip((a, b), outs, (s1, s2)):
            hs.attend_pages(c["shape"], *cu, o, lse, 0.1, stream=s)
    torch.cuda.synchronize()
    for c, (_, o, lse) in zip((a, b), outs):
        check(c, 0.1, got=(o.cpu().double(), lse.cpu().double()))


def test_results_repeat_bit_for_bit():
    c = case(1, 8, 8, 128, 16, 128, 128, [2048])
    first = run(c, 0.1)
    for _ in range(5):
        again = run(c, 0.1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


CAPTURED_FIRST = """
import sys, torch
sys.path[:0] = [sys.argv[1]]
import hierarchical_kv_cache_swap_gb300 as hs
from tests import page_models as pm
shape = (16, 2, 128)
pages = pm.random_pages(6, shape, 1).cuda().view(1, 6, -1)
k = torch.randn((5, 2, 128), device="cuda").to(torch.bfloat16)
dest = torch.arange(5, device="cuda")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
slots, sel, lengths = i32([[3, 0, 5]]), i32([[0, 1, 2]]), i32([44])
q = torch.randn((1, 1, 8, 128), device="cuda").to(torch.bfloat16)
o, lse = torch.zeros_like(q), torch.zeros((1, 1, 8), device="cuda")
ko = torch.zeros((1, 48, 2, 128), dtype=torch.bfloat16, device="cuda")
vo = torch.zeros_like(ko)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # the process's first calls
    hs.write_tokens(shape, k, k, dest, pages[0])
    hs.attend_pages(shape, q, pages, slots, sel, lengths, o, lse, 0.1)
    hs.read_pages(shape, pages, slots, ko, vo)
graph.replay()
torch.cuda.synchronize()
c, u = pm.quantise(k[:5].cpu())
ref = pages.cpu()
r, rl, to, tl = pm.attend(shape, q.cpu(), ref, slots.cpu(), sel.cpu(), lengths.cpu(), 0.1)
assert ((o.cpu().double() - r).abs() <= to).all() and ((lse.cpu().double() - rl).abs() <= tl).all()
kr = pm.read(ref[0], shape)[0][[3, 0, 5]].flatten(0, 1)
assert torch.equal(ko[0].cpu().double(), kr)
want = (pm.CODES[c].unflatten(-1, (-1, 16)) * pm.SCALES[u][..., None]).flatten(-2)
assert torch.equal(ko[0, 16:21].cpu().double(), want)
print("captured first: ok")
"""


def test_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURED_FIRST, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stdout + r.stderr


def test_calls_from_two_threads():
    cases = [case(2, 4, 8, 128, 16, 64, 64, [900, 1024], seed=s) for s in (1, 2)]
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got[i] = run(cases[i], 0.1, stream=s)

    ts = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for c, g in zip(cases, got):
        check(c, 0.1, got=g)


# ------------------------------------------------------------------ together, in a context
def test_decode_steps_over_a_paged_context():
    """Prompts stored into the host histories, then decode steps: each step's tokens join the
    histories (and the resident pages), the selected pages are resolved, read and attended."""
    shape, B, C, S, k, G = (16, 2, 128), 3, 24, 8, 6, 4
    T, H, D = shape
    E = hs.PageShape(*shape).bytes
    ctx = hs.Context(B, C, S, E)
    ctx.host_kv()[:] = 0
    hist = torch.zeros((B, C, E), dtype=torch.uint8)
    lens = [200, 33, 97]
    k0, v0 = tokens(sum(lens), H, D, torch.bfloat16, 1), tokens(sum(lens), H, D, torch.bfloat16, 2)
    req = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)])
    pos = torch.cat([torch.arange(n) for n in lens])
    ctx.append_tokens(shape, k0.cuda(), v0.cuda(), pos.int().cuda(), requests=req.int().cuda())
    torch.cuda.synchronize()
    pm.write(hist.view(B * C, E), shape, k0, v0, req * C * T + pos)
    assert torch.equal(torch.from_numpy(ctx.host_kv()[..., :E].copy()), hist)
    g = torch.Generator().manual_seed(4)
    for step in range(6):
        kn, vn = tokens(B, H, D, torch.bfloat16, 10 + step), tokens(B, H, D, torch.bfloat16, 20 + step)
        at = torch.tensor(lens, dtype=torch.int32)
        if step == 3:
            at[1] = -1  # no new token for this request
        ctx.append_tokens(shape, kn.cuda(), vn.cuda(), at.cuda())
        pm.write(hist.view(B * C, E), shape, kn, vn, torch.where(at >= 0, torch.arange(B) * C * T + at, -1))
        lens = [n + (a >= 0) for n, a in zip(lens, at.tolist())]
        sel = torch.full((B, k), -1, dtype=torch.int32)
        for b in range(B):
            held = -(-lens[b] // T)
            order = torch.randperm(held, generator=g)
            order = torch.cat([torch.tensor([held - 1]), order[order != held - 1]])[:k]
            sel[b, : len(order)] = order.int()
        out, miss = torch.empty((B, k), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        ctx.resolve(sel.cuda(), out, miss)
        q = torch.randn((B, 1, H * G, D), generator=g).to(torch.bfloat16)
        o, lse = torch.empty_like(q, device="cuda"), torch.empty((B, 1, H * G), device="cuda")
        lengths = torch.tensor(lens, dtype=torch.int32)
        ctx.attend_pages(shape, q.cuda(), out, sel.cuda(), lengths.cuda(), o, lse, D ** -0.5, softcap=30.0)
        ko = torch.empty((B, k * T, H, D), dtype=torch.bfloat16, device="cuda")
        vo = torch.empty_like(ko)
        ctx.read_pages(shape, out, ko, vo)
        torch.cuda.synchronize()
        assert ctx.status() == 0
        ro, rl, to, tl = pm.attend(shape, q, hist, sel, sel, lengths, D ** -0.5, cap=30.0)  # straight from the histories
        assert ((o.cpu().double() - ro).abs() <= to).all() and ((lse.cpu().double() - rl).abs() <= tl).all(), step
        want = torch.where((sel >= 0)[:, :, None, None, None],
                           pm.read(hist.view(B * C, E), shape)[1].view(B, C, T, H, D)[torch.arange(B)[:, None], sel.clamp(min=0).long()],
                           0.0).reshape(B, k * T, H, D)
        assert torch.equal(vo.cpu().double(), want)
    assert torch.equal(torch.from_numpy(ctx.host_kv()[..., :E].copy()), hist)
    # pages and requests that do not exist are skipped and reported
    before = ctx.host_kv().copy()
    bad = torch.tensor([C * T, 5, -1], dtype=torch.int32, device="cuda")
    ctx.append_tokens(shape, kn.cuda(), vn.cuda(), bad, requests=torch.tensor([0, B, 0], dtype=torch.int32, device="cuda"))
    assert ctx.status() == hs.HS_STATUS_RANGE and np.array_equal(ctx.host_kv(), before)
    with pytest.raises(hs.HsError):
        ctx.append_tokens(shape, kn[:2].cuda(), vn[:2].cuda(), bad[:2])  # two tokens for three requests
    with pytest.raises(hs.HsError):
        ctx.append_tokens((32, 2, 128), kn.cuda(), vn.cuda(), bad)  # not this context's pages
    ctx.close()


def test_tokens_join_extents_of_a_shared_pool():
    """Appended tokens land in each request's own extent of a pooled context's host store, and
    in its resident slots; pages past an extent are refused."""
    shape, rows, S, k = (32, 1, 64), 40, 4, 3
    T, H, D = shape
    E = hs.PageShape(*shape).bytes
    mem = torch.zeros(rows * E, dtype=torch.uint8).pin_memory()
    ctx = hs.Context(2, 16, S, E, pool=(mem.data_ptr(), rows, E))
    base, pages = [21, 3], [5, 9]
    ctx.set_extents(base, pages)
    ref = torch.zeros((rows, E), dtype=torch.uint8)
    n = [150, 288]
    req = torch.cat([torch.full((x,), b) for b, x in enumerate(n)])
    pos = torch.cat([torch.arange(x) for x in n])
    kk, vv = tokens(sum(n), H, D, torch.float16, 1), tokens(sum(n), H, D, torch.float16, 2)
    ctx.append_tokens(shape, kk.cuda(), vv.cuda(), pos.int().cuda(), requests=req.int().cuda())
    torch.cuda.synchronize()
    pm.write(ref, shape, kk, vv, torch.tensor(base)[req] * T + pos)
    assert torch.equal(mem.view(rows, E), ref) and ctx.status() == 0
    sel = torch.tensor([[4, 0, 2], [8, 1, 5]], dtype=torch.int32)
    out, miss = torch.empty((2, k), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    ctx.resolve(sel.cuda(), out, miss)
    # a token of a resident page is written in both places; one past the extent nowhere
    k1, v1 = tokens(2, H, D, torch.float16, 3), tokens(2, H, D, torch.float16, 4)
    ctx.append_tokens(shape, k1.cuda(), v1.cuda(), torch.tensor([5 * T, 8 * T + 31], dtype=torch.int32, device="cuda"))
    ctx.resolve(sel.cuda(), out, miss)
    q = torch.randn((2, 1, 3, D)).to(torch.float16)
    o, lse = torch.empty_like(q, device="cuda"), torch.empty((2, 1, 3), device="cuda")
    lengths = torch.tensor([150, 288], dtype=torch.int32)
    ctx.attend_pages(shape, q.cuda(), out, sel.cuda(), lengths.cuda(), o, lse, 0.2)
    torch.cuda.synchronize()
    assert ctx.status() == hs.HS_STATUS_RANGE and not miss.any()
    pm.write(ref, shape, k1[1:], v1[1:], torch.tensor([(base[1] + 8) * T + 31]))
    assert torch.equal(mem.view(rows, E), ref)
    hist = torch.stack([torch.nn.functional.pad(ref[b:b + x], (0, 0, 0, 16 - x)) for b, x in zip(base, pages)])
    ro, rl, to, tl = pm.attend(shape, q, hist, sel, sel, lengths, 0.2)
    for got, want, tol in ((o, ro, to), (lse, rl, tl)):  # the rows hold overflows: NaN blocks
        got, nan = got.cpu().double(), torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan) and ((got - want).abs()[~nan] <= tol[~nan]).all()
    ctx.close()


def test_attention_behind_a_resolution_in_chunks():
    """More requests than SMs: the resolution and its fetches are several overlapping kernels,
    and the attention launched behind them must see every page fetched."""
    shape, B, C, S, k = (16, 1, 64), 400, 12, 5, 4
    E = hs.PageShape(*shape).bytes
    ctx = hs.Context(B, C, S, E)
    hist = pm.random_pages(B * C, shape, 7).view(B, C, E)
    ctx.host_kv()[..., :E] = hist.numpy()
    g = torch.Generator().manual_seed(1)
    lengths = torch.full((B,), C * 16, dtype=torch.int32)
    q = torch.randn((B, 1, 2, 64), generator=g).to(torch.bfloat16)
    qd, ld = q.cuda(), lengths.cuda()
    sels = [torch.stack([torch.randperm(C, generator=g)[:k] for _ in range(B)]).int() for _ in range(6)]
    dev = [s.cuda() for s in sels]
    outs = []
    for s in dev:  # back to back, nothing waits in between
        out, miss = torch.empty((B, k), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        ctx.resolve(s, out, miss)
        o, lse = torch.empty_like(qd), torch.empty((B, 1, 2), device="cuda")
        ctx.attend_pages(shape, qd, out, s, ld, o, lse, 0.2)
        outs.append((o, lse))
    assert ctx.status() == 0
    for s, (o, lse) in zip(sels, outs):
        ro, rl, to, tl = pm.attend(shape, q, hist, s, s, lengths, 0.2)
        assert ((o.cpu().double() - ro).abs() <= to).all() and ((lse.cpu().double() - rl).abs() <= tl).all()
    ctx.close()


@pytest.mark.parametrize("captured", [False, True])
def test_pages_read_behind_a_resolution_whose_first_chunk_ends_last(captured):
    """The fetch of a later chunk, with nothing to copy, is done long before the first one's."""
    shape, B, C, k = (16, 4, 128), 320, 20, 16
    E = hs.PageShape(*shape).bytes
    ctx = hs.Context(B, C, k, E)
    ctx.host_kv()[..., :E] = pm.random_pages(C, shape, 3).numpy()
    sel = torch.full((B, k), -1, dtype=torch.int32)
    sel[:B // 3] = torch.arange(k, dtype=torch.int32) + 2
    sel, out = sel.cuda(), torch.full((B, k), -1, dtype=torch.int32, device="cuda")
    miss = torch.empty(B, dtype=torch.int32, device="cuda")
    k1, v1, k2, v2 = (torch.empty((B, k * 16, 4, 128), dtype=torch.float16, device="cuda") for _ in range(4))

    def step():
        ctx.resolve(sel, out, miss)
        ctx.read_pages(shape, out, k1, v1)

    if captured:
        ctx.read_pages(shape, out, k1, v1)  # loads the kernel
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            step()
        step = graph.replay
    ctx.device_kv().zero_()
    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    ctx.read_pages(shape, out, k2, v2)
    assert ctx.status() == 0 and int(miss.sum()) == B // 3 * k
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    n = k * 16
    got = torch.stack([k2[0].cpu(), k2[B // 3 - 1].cpu()])
    assert torch.equal(got[0], got[1]) and bool((got[0].abs().amax(dim=(1, 2)) > 0).all()) and got.shape[1] == n
    ctx.close()

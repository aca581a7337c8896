"""Latent entries, the absorbed form's products and prompts' attention on the GPU, against the 64-bit
models of tests/latent_models.py: written codes and read values are equal, sums within derived bounds."""
import math
import os
import subprocess
import sys

import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import latent_models as lm

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ entries
def tokens(n, dtype, seed):
    """Latents of very different sizes, with exact ties, zeros and signed zeros among them."""
    g = gen(seed)
    x = normal(g, n, 4, 128) * torch.exp(4 * normal(g, n, 4, 1))
    ties = torch.randint(-464, 465, (n, 4, 128), generator=g, device="cuda").float()
    x = torch.where(torch.rand((n, 4, 1), generator=g, device="cuda") < 0.4, ties, x).view(n, 512)
    x[torch.rand((n, 512), generator=g, device="cuda") < 0.05] = -0.0
    return x.to(dtype), normal(g, n, 64).to(dtype)


def check_entries(got, latent, rope, want_rope):
    """Entries [n, 656]: codes and scales equal, rotary keys off by an f32 rotation and one rounding."""
    c, s, bad = lm.codes(latent)
    assert torch.equal(got[:, :512][~bad], c[~bad])
    sg = got[:, 512:528].contiguous().view(torch.float32).double()
    assert torch.equal(torch.isnan(sg), torch.isnan(s)) and torch.equal(sg.nan_to_num(), s.nan_to_num())
    r = got[:, 528:].contiguous().view(BF16).double()
    size = rope.double().abs().amax(-1, keepdim=True) if rope.numel() else 0
    assert ((r - want_rope).abs() <= 2.0 ** -8 * want_rope.abs() + 6 * lm.EPS32 * size + 2.0 ** -133).all()


@pytest.mark.parametrize("n,dtype,halves,turned", [
    (1, BF16, False, True), (64, BF16, False, True), (37, F16, True, True), (1021, BF16, True, True), (300, F16, False, False),
    (5, BF16, True, False), (0, BF16, False, True)])
def test_written_entries_and_read_values(n, dtype, halves, turned):
    latent, rope = tokens(n, dtype, n)
    N = n + 5
    entries = torch.randint(0, 256, (N, 656), dtype=torch.uint8, device="cuda", generator=gen(1))
    before = entries.clone()
    place = torch.randperm(N, generator=gen(2), device="cuda")[:n]
    dest = place.clone()
    dest[3::7] = -1 - dest[3::7]  # padding
    tab = lm.table(50).cuda()
    pos = torch.randint(0, 50, (n,), dtype=torch.int32, device="cuda", generator=gen(3))
    word = status_word()
    turn = dict(rotation=tab, positions=pos, halves=halves) if turned else {}
    hs.write_latents(latent, rope, dest, entries, status=word, **turn)
    want = lm.rotate(rope, tab, pos, halves) if turned else rope.double()
    live = dest >= 0
    check_entries(entries[place[live]], latent[live], rope[live], want[live])
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[place[live]] = False
    assert torch.equal(entries[rest], before[rest])
    slots = place.to(torch.int32).view(1, n).clone()
    slots[0, 1::5] = -1
    for out in (BF16, F16):
        lo = torch.full((1, n, 512), 7.0, dtype=out, device="cuda")
        ro = torch.full((1, n, 64), 7.0, dtype=out, device="cuda")
        hs.read_latents(entries.view(1, N, 656), slots, lo, ro, status=word)
        lv, rv = lm.values(entries[place])
        lv[slots[0] < 0], rv[slots[0] < 0] = 0, 0
        keep = live | (slots[0] < 0)  # the others hold random bytes
        for got, ref in ((lo[0][keep], lv[keep].to(out)), (ro[0][keep], rv[keep].to(out))):
            assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got[~torch.isnan(ref)], ref[~torch.isnan(ref)])
    assert int(word) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_every_magnitude_as_a_blocks_largest(dtype):
    """Each positive number of the type (infinities and NaNs too) as the largest of a block, beside
    fractions of it."""
    a = torch.arange(0, 32768, dtype=torch.int16).view(dtype).cuda()
    x = torch.zeros((32768, 128), dtype=dtype, device="cuda")
    x[:, 0], x[:, 3] = a, -(a.float() / 2).to(dtype)
    for i in range(4, 128):
        x[:, i] = (a.float() * (i / 128.0)).to(dtype)
    latent = x.view(8192, 512)
    entries = torch.zeros((8192, 656), dtype=torch.uint8, device="cuda")
    rope = torch.zeros((8192, 64), dtype=dtype, device="cuda")
    hs.write_latents(latent, rope, torch.arange(8192, device="cuda"), entries)
    c, s, bad = lm.codes(latent)
    got = entries[:, 512:528].contiguous().view(torch.float32).double()
    assert torch.equal(torch.isnan(got), torch.isnan(s)) and torch.equal(got.nan_to_num(), s.nan_to_num())
    assert torch.equal(entries[:, :512][~bad], c[~bad])
    lo = torch.empty((1, 8192, 512), dtype=BF16, device="cuda")
    ro = torch.empty((1, 8192, 64), dtype=BF16, device="cuda")
    hs.read_latents(entries.view(1, -1, 656), torch.arange(8192, dtype=torch.int32, device="cuda").view(1, -1), lo, ro)
    assert torch.equal(torch.isnan(lo[0]), bad)


def test_strided_rows_and_rows_out_of_range():
    n = 40
    wide = normal(gen(5), n, 1024).to(BF16)
    latent, rope = wide[:, 8:520], wide[:, 528:592]
    tab = lm.table(10).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda") % 12 - 1  # -1 and 10 have no row
    dest = torch.arange(n, device="cuda")
    dest[7], dest[8] = n, 1 << 40
    entries = torch.zeros((n, 656), dtype=torch.uint8, device="cuda")
    word = status_word()
    hs.write_latents(latent, rope, dest, entries, rotation=tab, positions=pos, status=word)
    assert int(word) == hs.HS_STATUS_RANGE
    live = (pos >= 0) & (pos < 10) & (dest < n)
    check_entries(entries[live], latent[live], rope[live], lm.rotate(rope[live], tab, pos[live], False))
    assert not entries[~live].any()
    word.zero_()
    slots = torch.tensor([[0, n, -5], [1, 2, 1 << 30]], dtype=torch.int32, device="cuda")
    lo, ro = torch.ones((2, 3, 512), dtype=BF16, device="cuda"), torch.ones((2, 3, 64), dtype=BF16, device="cuda")
    hs.read_latents(entries.view(2, n // 2, 656), slots, lo, ro, status=word)
    assert int(word) == hs.HS_STATUS_RANGE
    assert not lo[0, 1:].any() and not lo[1, 2].any() and not ro[0, 1:].any()
    assert torch.equal(lo[1, 0].double(), lm.values(entries[n // 2 + 1])[0])


def test_entries_in_pinned_memory():
    n = 19
    latent, rope = tokens(n, BF16, 3)
    entries = torch.zeros((n, 656), dtype=torch.uint8).pin_memory()
    hs.write_latents(latent, rope, torch.arange(n, device="cuda"), entries)
    torch.cuda.synchronize()
    check_entries(entries.cuda(), latent, rope, rope.double())


@pytest.mark.parametrize("pooled", [False, True])
def test_appended_latents(pooled):
    """Tokens into histories: padding, requests and positions out of range, a resident one rewritten."""
    R, C, S, n = 3, 20, 8, 26
    word = hs.HS_STATUS_RANGE
    if pooled:
        store = torch.zeros((64, 656), dtype=torch.uint8).pin_memory()
        ctx = hs.Context(R, C, S, 656, pool=(store.data_ptr(), 64, 656))
        base, length = [40, 0, 21], [20, 13, 0]
        ctx.set_extents(base, length)
    else:
        ctx = hs.Context(R, C, S, 656)
        base, length = [0, C, 2 * C], [C] * 3
    host = ctx.host_kv().reshape(-1, ctx.host_stride)
    host[:] = 3
    latent, rope = tokens(n, BF16, 4)
    tab = lm.table(C + 3, 2).cuda()
    req = torch.arange(n, dtype=torch.int32) % 3
    pos = torch.arange(n, dtype=torch.int32) // 3
    req[5], req[6], pos[7], pos[8], pos[9] = -1, R, -4, C, C - 1
    turn = pos.clamp(min=0, max=C + 2) * 0 + torch.arange(n, dtype=torch.int32) % (C + 3)
    turn[10] = C + 3  # no row
    ctx.append_latents(latent, rope, pos.cuda(), requests=req.cuda(), rotation=tab, rotation_positions=turn.cuda())
    assert ctx.status() == word
    want = lm.rotate(rope, tab, turn.cuda().clamp(max=C + 2), False)
    seen = set()
    got = torch.from_numpy(host).cuda()
    for i in range(n):
        r, p = int(req[i]), int(pos[i])
        if r < 0 or r >= R or p < 0 or p >= length[r] or i == 10:
            continue
        seen.add(base[r] + p)
        check_entries(got[base[r] + p][None, :656], latent[i:i + 1], rope[i:i + 1], want[i:i + 1])
    rest = [i for i in range(host.shape[0]) if i not in seen]
    assert len(seen) >= 12 and (host[rest][:, :656] == 3).all()
    ctx.clear_status()
    # resident entries are rewritten in their slots, in fp16 and with halves this time
    sel = torch.tensor([[0, 1, 2], [3, 2, 0], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    slots, miss = torch.empty_like(sel), torch.empty(R, dtype=torch.int32, device="cuda")
    ctx.resolve(sel, slots, miss)
    latent, rope = tokens(R, F16, 5)
    ctx.append_latents(latent, rope, torch.tensor([1, 3, -1], dtype=torch.int32, device="cuda"), rotation=tab, halves=True)
    lo, ro = torch.empty((R, 3, 512), dtype=BF16, device="cuda"), torch.empty((R, 3, 64), dtype=BF16, device="cuda")
    ctx.read_latents(slots, lo, ro)
    assert ctx.status() == 0
    got = torch.from_numpy(host).cuda()
    want = lm.rotate(rope, tab, torch.tensor([1, 3, 0], device="cuda"), True)
    for r, p, j in ((0, 1, 1), (1, 3, 0)):
        check_entries(got[base[r] + p][None, :656], latent[r:r + 1], rope[r:r + 1], want[r:r + 1])
        a, b = lm.values(got[base[r] + p][:656])
        assert torch.equal(lo[r, j], a.to(BF16)) and torch.equal(ro[r, j].double(), b)
    assert not lo[2].any()
    ctx.close()


# ------------------------------------------------------------------------ the absorbed form
@pytest.mark.parametrize("n,H,halves,turned", [(1, 128, False, True), (1, 1, True, True), (16, 3, True, True), (17, 5, False, True),
                                               (37, 20, True, True), (64, 16, False, True), (65, 2, False, False), (256, 8, False, True),
                                               (300, 1, True, True), (0, 4, False, True)])
def test_products_of_the_absorbed_form(n, H, halves, turned):
    g = gen(n * 131 + H)
    q = normal(g, n, H + 1, 200).to(BF16)[:, 1:, :192]  # strided
    both = (normal(g, H, 256, 512) * 512 ** -0.5).to(BF16)
    tab = lm.table(33).cuda()
    pos = torch.randint(0, 33, (n,), dtype=torch.int32, device="cuda", generator=g)
    pos[2::5] = -3  # padding
    out = torch.full((n, H, 576), 7.0, dtype=BF16, device="cuda")
    word = status_word()
    hs.absorb_queries(q, both[:, :128], out, status=word, **(dict(rotation=tab, positions=pos, halves=halves) if turned else {}))
    ref = torch.einsum("nhd,hdc->nhc", q[..., :128].double(), both[:, :128].double())
    size = torch.einsum("nhd,hdc->nhc", q[..., :128].double().abs(), both[:, :128].double().abs())
    assert ((out[..., :512].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 130 * 2.0 ** -23 * size).all()
    want = q[..., 128:].double()
    if turned:
        want = lm.rotate(q[..., 128:], tab, pos.clamp(min=0), halves)
        want[pos < 0] = 0
    assert ((out[..., 512:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 6 * lm.EPS32 * 8).all()
    assert int(word) == 0

    o = (normal(g, n, H, 520) * torch.exp(2 * normal(g, n, H, 1)))[..., 4:516]
    back = torch.full((n, H, 128), 7.0, dtype=BF16, device="cuda")
    hs.expand_outputs(o, both[:, 128:], back)
    ref = torch.einsum("nhc,hec->nhe", o.double(), both[:, 128:].double())
    size = torch.einsum("nhc,hec->nhe", o.double().abs(), both[:, 128:].double().abs())
    assert ((back.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 514 * 2.0 ** -23) * size).all()


def test_queries_whose_positions_have_no_row():
    q = normal(gen(1), 3, 2, 192).to(BF16)
    up = normal(gen(2), 2, 128, 512).to(BF16)
    out = torch.ones((3, 2, 576), dtype=BF16, device="cuda")
    word = status_word()
    hs.absorb_queries(q, up, out, rotation=lm.table(4).cuda(), positions=torch.tensor([0, 4, 3], dtype=torch.int32, device="cuda"), status=word)
    assert int(word) == hs.HS_STATUS_RANGE and not out[1, :, 512:].any() and out[0, :, 512:].any()


# ------------------------------------------------------------------------ prompts
def prompts(lens, H, dtype, seed, first=(0, 0), behind=(0, 0)):
    """Tensors of prompts of (query, key) counts, `first` rows before them and `behind` after them, in
    strided views; the rows outside are NaN."""
    g = gen(seed)
    nq, nk = (first[i] + sum(x[i] for x in lens) + behind[i] for i in (0, 1))
    q = normal(g, nq, H, 200).to(dtype)[..., 8:]
    kv = normal(g, nk, H, 256).to(dtype)
    r = normal(g, nk, 72).to(dtype)[:, :64]
    for x, i in ((q, 0), (kv, 1), (r, 1)):
        x[:first[i]] = math.nan
        x[x.shape[0] - behind[i]:] = math.nan
    starts = [torch.tensor([first[i] + sum(x[i] for x in lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
              for i in (0, 1)]
    return q, kv[..., :128], r, kv[..., 128:], *starts


def check_prompts(lens, H, dtype, causal, args, scale=192 ** -0.5, **kw):
    q, k, r, v, qs, ks = args
    o = torch.full((q.shape[0], H, 136), 7.0, dtype=dtype, device="cuda")[..., :128]
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    word = status_word()
    hs.attend_prompts(q, k, r, v, qs, ks, o, lse, scale, causal=causal, status=word, **kw)
    assert int(word) == 0
    outside = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    for b, (lq, lk) in enumerate(lens):
        a, c = int(qs[b]), int(ks[b])
        outside[a:a + lq] = False
        wo, wl, bo, bl = lm.attend(q[a:a + lq], k[c:c + lk], r[c:c + lk], v[c:c + lk], scale, causal, dtype)
        assert lm.near(o[a:a + lq], wo, bo), (b, lq, lk, (o[a:a + lq].double() - wo).abs().max())
        assert lm.near(lse[a:a + lq], wl, bl), (b, lq, lk, (lse[a:a + lq].double() - wl).abs().max())
    assert (o[outside] == 7).all() and (lse[outside] == 7).all()
    return o, lse


@pytest.mark.parametrize("lens,H,dtype,causal", [
    ([(1, 1)], 1, BF16, True), ([(128, 128)], 1, BF16, False), ([(77, 77)], 3, BF16, True), ([(256, 256)], 2, F16, True),
    ([(129, 129), (1, 300), (0, 5), (40, 40), (300, 1)], 2, BF16, True), ([(257, 1000)], 2, F16, True),
    ([(5, 0), (0, 0), (130, 64), (64, 129)], 2, BF16, False), ([(200, 17), (17, 200)], 1, F16, True),
    ([(1, 2049)], 16, BF16, True), ([(600, 1500), (700, 640)], 4, BF16, True), ([(1, 1)] * 70, 2, BF16, True),
    ([(13, 40)] * 33 + [(300, 300)], 1, F16, False), ([], 3, BF16, True), ([(3, 0)], 2, BF16, True)])
def test_prompts(lens, H, dtype, causal):
    check_prompts(lens, H, dtype, causal, prompts(lens, H, dtype, len(lens) + H, first=(3, 2), behind=(9, 150)))


@pytest.mark.parametrize("most,H", [(100, 16), (300, 8), (700, 5)])
def test_many_prompts(most, H):
    """More tiles than run at once, whose second half, keys or all rows may be missing."""
    g = torch.Generator().manual_seed(most)
    n = 160
    lens = [(most, most)] * n if most == 100 else [
        tuple((torch.rand(2, generator=g) * most).int().tolist()) if i % 3 else (int(most * float(torch.rand(1, generator=g))), 0 if i % 2 else 129)
        for i in range(n)]
    check_prompts(lens, H, BF16, True, prompts(lens, H, BF16, most))


def test_prompts_whose_tensors_end_with_them():
    lens = [(100, 140), (129, 257)]
    check_prompts(lens, 3, BF16, True, prompts(lens, 3, BF16, 5))


def test_prompts_without_any_key():
    lens = [(3, 0), (140, 0)]
    check_prompts(lens, 2, BF16, True, prompts(lens, 2, BF16, 5))


@pytest.mark.parametrize("scale", [1e-6, 0.5, 30.0])
def test_prompts_of_small_and_large_scores(scale):
    lens = [(150, 400), (33, 33)]
    check_prompts(lens, 2, BF16, True, prompts(lens, 2, BF16, 8), scale=scale)


def test_scores_that_rise_along_the_keys():
    """The maximum moves at every tile."""
    lens = [(128, 1024)]
    q, k, r, v, qs, ks = prompts(lens, 1, BF16, 9)
    q.abs_()
    k.copy_((torch.arange(1024, device="cuda")[:, None, None] / 64.0 * torch.ones_like(k)).to(BF16))
    check_prompts(lens, 1, BF16, False, (q, k, r, v, qs, ks), scale=0.05)


def test_prompts_starts_out_of_order_or_range():
    lens = [(40, 40), (50, 50), (60, 60)]
    for bad in (0, 1):
        q, k, r, v, *starts = prompts(lens, 2, BF16, 11)
        full = [s.clone() for s in starts]
        starts[bad][3] = 10 ** 6
        o, lse = torch.full((150, 2, 128), 7.0, dtype=BF16, device="cuda"), torch.full((150, 2), 7.0, device="cuda")
        word = status_word()
        hs.attend_prompts(q, k, r, v, *starts, o, lse, 0.1, status=word)
        assert int(word) == hs.HS_STATUS_RANGE
        ref, rl = torch.empty_like(o), torch.empty_like(lse)
        hs.attend_prompts(q, k, r, v, *full, ref, rl, 0.1)
        assert torch.equal(o[:90], ref[:90]) and (o[90:] == 7).all() and torch.equal(lse[:90], rl[:90])
    starts[0][1], starts[0][2] = 30, 20  # descending
    word = status_word()
    starts[1].copy_(full[1])
    hs.attend_prompts(q, k, r, v, *starts, o, lse, 0.1, status=word)
    assert int(word) == hs.HS_STATUS_RANGE


# ------------------------------------------------------------------------ streams and graphs
def test_a_captured_and_replayed_layer():
    """Every call on a side stream, captured once and replayed over new inputs."""
    H, n = 4, 6
    latent, rope = tokens(n, BF16, 1)
    tab = lm.table(64).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    entries = torch.zeros((n, 656), dtype=torch.uint8, device="cuda")
    lo, ro = torch.zeros((1, n, 512), dtype=BF16, device="cuda"), torch.zeros((1, n, 64), dtype=BF16, device="cuda")
    q, both = normal(gen(1), n, H, 192).to(BF16), normal(gen(2), H, 256, 512).to(BF16)
    qo, x, back = torch.zeros((n, H, 576), dtype=BF16, device="cuda"), normal(gen(3), n, H, 512), torch.zeros((n, H, 128), dtype=BF16, device="cuda")
    k = normal(gen(4), n, H, 128).to(BF16)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    po, pl = torch.zeros_like(back), torch.zeros((n, H), device="cuda")
    dest, slots = torch.arange(n, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)

    def layer():
        hs.write_latents(latent, rope, dest, entries, rotation=tab, positions=pos)
        hs.read_latents(entries.view(1, n, 656), slots, lo, ro)
        hs.absorb_queries(q, both[:, :128], qo, rotation=tab, positions=pos)
        hs.expand_outputs(x, both[:, 128:], back)
        hs.attend_prompts(q, k, ro[0], k, starts, starts, po, pl, 0.1)

    outs = (entries, lo, ro, qo, back, po, pl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer()
    for seed in (7, 8):
        g = gen(seed)
        for t in (latent, rope, q, x, k):
            t.copy_(normal(g, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))


FIRST = """
import torch, hierarchical_kv_cache_swap_gb300 as hs
z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
lat, rope, ent, dest = z(3, 512), z(3, 64), z(4, 656, t=torch.uint8), torch.arange(3, device="cuda")
slots, q, up, qo, o, oo = dest.int().view(1, 3), z(40, 2, 192) + 1, z(2, 128, 512) + 1, z(40, 2, 576), z(40, 2, 512, t=torch.float32) + 1, z(40, 2, 128)
many = z(200, 128, 512, t=torch.float32) + 1, z(128, 128, 512) + 1, z(200, 128, 128)
starts, po, pl = torch.tensor([0, 40], dtype=torch.int32, device="cuda"), z(40, 2, 128), z(40, 2, t=torch.float32)
k = z(40, 2, 128) + 1
torch.cuda.synchronize()
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(side):
    graph.capture_begin()
    hs.write_latents(lat + 1, rope, dest, ent)
    hs.read_latents(ent[None], slots, lat[None], rope[None])
    hs.absorb_queries(q, up, qo)
    hs.expand_outputs(o, up, oo)
    hs.expand_outputs(*many)
    hs.attend_prompts(q, k, z(40, 64), k, starts, starts, po, pl, 0.1)
    graph.capture_end()
graph.replay()
torch.cuda.synchronize()
assert (lat == 1).all() and (qo[..., :512] == 128).all() and (oo == 512).all() and (many[2] == 512).all() and (po == 1).all()
"""


def test_first_calls_of_a_process_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST], cwd=root, check=True, timeout=200)


def test_calls_on_two_streams_at_once():
    """Nothing is shared between calls: each stream's results are those of its call alone."""
    H, lens = 8, [(700, 900), (33, 33), (129, 400)]
    sets = [prompts(lens, H, BF16, seed) for seed in (1, 2)]
    n = 300
    more = [(normal(gen(s), n, H, 192).to(BF16), normal(gen(s + 5), H, 256, 512).to(BF16), normal(gen(s + 9), n, H, 512)) for s in (3, 4)]
    rows = sets[0][0].shape[0]

    def outs():
        return (torch.zeros((rows, H, 128), dtype=BF16, device="cuda"), torch.zeros((rows, H), device="cuda"),
                torch.zeros((n, H, 576), dtype=BF16, device="cuda"), torch.zeros((n, H, 128), dtype=BF16, device="cuda"))

    def calls(i, to, stream=None):
        q, k, r, v, qs, ks = sets[i]
        x, both, o = more[i]
        hs.attend_prompts(q, k, r, v, qs, ks, to[0], to[1], 0.1, stream=stream)
        hs.absorb_queries(x, both[:, :128], to[2], stream=stream)
        hs.expand_outputs(o, both[:, 128:], to[3], stream=stream)

    want = [outs(), outs()]
    for i in (0, 1):
        calls(i, want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [outs(), outs()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            calls(i, got[i], streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in (0, 1) for a, b in zip(got[i], want[i]))


# ------------------------------------------------------------------------ a layer of a model
def test_prompts_join_the_histories_and_are_decoded_absorbed():
    """Prompts are attended in the expanded form and appended; then a token of each request is
    decoded in the absorbed form: appended, resolved, its queries absorbed, attended, its output
    expanded. The expanded form over the entries read back gives the same."""
    R, C, H, lens = 3, 300, 16, [200, 1, 77]
    g = gen(21)
    up = (normal(g, H, 256, 512) * 512 ** -0.5).to(BF16)
    tab, scale = lm.table(C, 4).cuda(), 192 ** -0.5
    ctx = hs.Context(R, C, 256, 656)
    n = sum(lens)
    latent, rope = normal(g, n, 512).to(BF16), normal(g, n, 64).to(BF16)
    pos = torch.cat([torch.arange(x, dtype=torch.int32) for x in lens]).cuda()
    req = torch.cat([torch.full((x,), i, dtype=torch.int32) for i, x in enumerate(lens)]).cuda()
    ctx.append_latents(latent, rope, pos, requests=req, rotation=tab)
    new_l, new_r = normal(g, R, 512).to(BF16), normal(g, R, 64).to(BF16)
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ctx.append_latents(new_l, new_r, at, rotation=tab)
    k = 201
    sel = torch.full((R, k), -1, dtype=torch.int32, device="cuda")
    for i, x in enumerate(lens):
        sel[i, :x + 1] = torch.arange(x + 1, dtype=torch.int32, device="cuda")
    slots, miss = torch.empty_like(sel), torch.empty(R, dtype=torch.int32, device="cuda")
    ctx.resolve(sel, slots, miss)
    assert miss.tolist() == [x + 1 for x in lens]
    # a rewrite of a resident token reaches its slot
    ctx.append_latents(new_l, new_r, at, rotation=tab)
    q = normal(g, R, H, 192).to(BF16)
    qa = torch.empty((R, H, 576), dtype=BF16, device="cuda")
    hs.absorb_queries(q, up[:, :128], qa, rotation=tab, positions=at)
    o, lse = torch.empty((R, H, 512), device="cuda"), torch.empty((R, H), device="cuda")
    nbytes = ctx.attend_workspace(R, H, k)
    ctx.attend(qa, slots, o, lse, scale, workspace=torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda") if nbytes else None)
    out = torch.empty((R, H, 128), dtype=BF16, device="cuda")
    hs.expand_outputs(o, up[:, 128:], out)

    lo, ro = torch.empty((R, k, 512), dtype=BF16, device="cuda"), torch.empty((R, k, 64), dtype=BF16, device="cuda")
    ctx.read_latents(slots, lo, ro)
    assert ctx.status() == 0
    c, s, _ = lm.codes(torch.cat((latent, new_l)))
    host = torch.from_numpy(ctx.host_kv()).cuda()
    for i, x in enumerate(lens):
        first = sum(lens[:i])
        rows = list(range(first, first + x)) + [n + i]
        check_entries(host[i, :x + 1, :656], torch.cat((latent, new_l))[rows], torch.cat((rope, new_r))[rows],
                      lm.rotate(torch.cat((rope, new_r))[rows], tab, torch.arange(x + 1, device="cuda"), False))
        assert torch.equal(lo[i, :x + 1].double(), lm.values(host[i, :x + 1, :656])[0])
    # the same in 64 bits, from the entries
    qr = lm.rotate(q[..., 128:], tab, at, False)
    for i, x in enumerate(lens):
        lat, rk = lo[i, :x + 1].double(), ro[i, :x + 1].double()
        kk, vv = torch.einsum("tc,hdc->thd", lat, up[:, :128].double()), torch.einsum("tc,hdc->thd", lat, up[:, 128:].double())
        y = (torch.einsum("hd,thd->ht", q[i, :, :128].double(), kk) + torch.einsum("hd,td->ht", qr[i], rk)) * scale
        w = torch.softmax(y, -1)
        ref = torch.einsum("ht,thd->hd", w, vv)
        # the absorbed query is rounded (2^-8 of |q'| |latent| in each score), so are the weights, o and out
        err = 2.0 ** -8 * torch.einsum("hc,tc->ht", torch.einsum("hd,hdc->hc", q[i, :, :128].double(), up[:, :128].double()).abs(), lat.abs()) * scale
        err = err + 2.0 ** -8 * torch.einsum("hd,td->ht", qr[i].abs(), rk.abs()) * scale
        size = torch.einsum("ht,thd->hd", w, vv.abs())
        deep = torch.einsum("ht,tc,hec->he", w, lat.abs(), up[:, 128:].double().abs())
        assert ((out[i].double() - ref).abs() <= 2 * err.amax() * size + 2.0 ** -7 * deep + 2.0 ** -8 * ref.abs()).all()
        assert ((lse[i].double() - torch.logsumexp(y, -1)).abs() <= err.amax() + 2.0 ** -8).all()
    # the prompts' last tokens in the expanded form, keys and values by a product of the library
    kv = torch.cat([lo[i, :x + 1] for i, x in enumerate(lens)]) @ up.view(-1, 512).T
    kv = kv.view(-1, H, 256)
    rr = torch.cat([ro[i, :x + 1] for i, x in enumerate(lens)]).contiguous()
    qx = torch.cat((q[..., :128], qr.to(BF16)), -1)
    qs = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    ks = torch.tensor([0, *torch.tensor([x + 1 for x in lens]).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    po, pl = torch.empty((R, H, 128), dtype=BF16, device="cuda"), torch.empty((R, H), device="cuda")
    hs.attend_prompts(qx, kv[..., :128], rr, kv[..., 128:], qs, ks, po, pl, scale)
    assert ((po.double() - out.double()).abs() <= 0.05 * out.double().abs() + 0.02).all()
    assert ((pl - lse).abs() <= 0.05).all()
    ctx.close()

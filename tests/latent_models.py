"""64-bit models of the latent operators, written from their definitions, with the bounds of
what the kernels' roundings may change. A rounding to a type is off by at most half a step,
finfo.eps / 2 of the value."""
import math

import torch

LATENT, ROPE, HEAD, ENTRY = 512, 64, 128, 656
EPS32 = 2.0 ** -24
# the E4M3 numbers of codes 0 .. 127
LEVELS = [(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)] + [math.nan]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def table(rows, seed=0):
    """Cosines and sines of `rows` positions, fp32 [rows, 64]."""
    g = torch.Generator().manual_seed(seed)
    angle = torch.rand((rows, 32), generator=g, dtype=torch.float64) * 2 * math.pi
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def rotate(x, tab, positions, halves):
    """x [n, ..., 64] rotated in 64 bits, row i by positions[i]."""
    t = tab.double()[positions.long()].view(-1, *(1,) * (x.dim() - 2), ROPE)
    c, s = t[..., :32], t[..., 32:]
    x, y = x.double(), torch.empty(x.shape, dtype=torch.float64, device=x.device)
    a, b = (slice(0, 32), slice(32, 64)) if halves else (slice(0, 64, 2), slice(1, 64, 2))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def scales(x):
    """The scales [n, 4] of latents x [n, 512]: the smallest power of two s >= 2^-126 with 448 s >= max |x|."""
    big = x.double().abs().unflatten(-1, (4, 128)).amax(-1)
    powers = torch.tensor([2.0 ** e for e in range(-126, 128)], dtype=torch.float64, device=x.device)
    s = powers[torch.searchsorted(448 * powers, torch.where(torch.isfinite(big), big, 0.0).contiguous())]
    return torch.where(torch.isfinite(big), s, math.nan)


def codes(x):
    """The E4M3 codes [n, 512] and the scales of latents x."""
    s = scales(x)
    level = torch.tensor(LEVELS[:127], dtype=torch.float64, device=x.device)
    y = (x.double().unflatten(-1, (4, 128)) / s[..., None]).flatten(-2)
    bad = torch.isnan(y)
    m = torch.where(bad, 0.0, y.abs())
    hi = torch.searchsorted(level, m).clamp(1, 126)
    up, down = level[hi] - m, m - level[hi - 1]
    c = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return (c + 128 * torch.signbit(y)).to(torch.uint8), s, bad


def values(entries):
    """What entries [..., 656] stand for: latents and rotary keys, 64 bits."""
    v = torch.tensor(LEVELS + [-x for x in LEVELS], dtype=torch.float64, device=entries.device)[entries[..., :512].long()]
    s = entries[..., 512:528].contiguous().view(torch.float32).double()
    return (v.unflatten(-1, (4, 128)) * s[..., None]).flatten(-2), entries[..., 528:].contiguous().view(torch.bfloat16).double()


def attend(q, k, r, v, scale, causal, dtype):
    """One prompt: q [Lq, H, 192], k and v [Lk, H, 128], r [Lk, 64]. o, lse and their bounds.

    A score's products of 16-bit floats are exact in f32; their sum of 192 terms, scaled, is off by at
    most e = 200 * 2^-23 of the sum of the magnitudes (an addition may truncate), and the exponent's
    subtraction by 2^-22 of the largest |s| more; exp2 by 2^-21. A weight is so off by e' = 2 (e + ...)
    relative to the weights' sum and rounded to `dtype` (in fp16 by 2^-25 of the largest at the least,
    which is at least 1 against the kept maximum); sums of n terms by n 2^-23; the result is rounded."""
    q, k, r, v = (x.double() for x in (q, k, r, v))
    Lq, Lk = q.shape[0], k.shape[0]
    if Lq == 0 or Lk == 0:
        o = torch.zeros((Lq, q.shape[1], HEAD), dtype=torch.float64, device=q.device)
        return o, torch.full_like(o[..., 0], -math.inf), o, o[..., 0]
    kk = torch.cat((k, r[:, None].expand(-1, q.shape[1], -1)), -1)
    x = torch.einsum("qhd,khd->hqk", q, kk) * scale
    size = torch.einsum("qhd,khd->hqk", q.abs(), kk.abs()).nan_to_num() * scale
    see = torch.ones((Lq, Lk), dtype=torch.bool, device=q.device)
    if causal:
        see = torch.arange(Lk, device=q.device) <= torch.arange(Lq, device=q.device)[:, None] + (Lk - Lq)
    x = torch.where(see, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    safe = torch.where(top > -math.inf, top, 0.0)
    w = torch.where(see, torch.exp(x - safe), 0.0)
    total = w.sum(-1, keepdim=True)
    empty = ~see.any(-1)
    w = w / torch.where(total != 0, total, 1.0)
    vz = [torch.where(see[i][:, None, None], v, 0.0) for i in range(Lq)] if not torch.isfinite(v).all() else None
    if vz is None:
        o = torch.einsum("hqk,khd->qhd", w, v)
    else:
        o = torch.stack([torch.einsum("hk,khd->hd", w[:, i], vz[i]) for i in range(Lq)])
    lse = (torch.log(total) + safe)[..., 0].transpose(0, 1)
    e = 200 * 2.0 ** -23 * size.amax((1, 2), keepdim=True) + 2.0 ** -22 * (x.abs().nan_to_num(nan=0.0, posinf=0.0).amax((1, 2), keepdim=True) + 8)
    e = (2 * e + 2.0 ** -20)
    absw = torch.einsum("hqk,khd->qhd", w.nan_to_num(), v.abs().nan_to_num(posinf=0.0))
    u = half_step(dtype)
    bound = (2 * e.view(1, -1, 1) + u + (Lk + 16) * 2.0 ** -23) * absw + u * o.abs() + 1e-30
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25 * v.abs().nan_to_num(posinf=0.0).sum(0)
    else:
        bound = bound + 2.0 ** -133
    o[empty], lse[empty] = 0.0, -math.inf
    return o, lse, bound, e.view(1, -1) + 2.0 ** -19 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


def near(got, want, bound):
    """got is within bound of want, and not finite where want is not."""
    got = got.double()
    fine = torch.isfinite(want)
    same = torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    return same and bool(((got - want).abs() <= bound)[fine].all())

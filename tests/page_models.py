"""4-bit pages and the attention over them, plainly and in 64 bits, from the definitions in
include/hs.h. Shares nothing with the kernels: codes and scales are found by search in the
tables of the values they stand for, pages are assembled byte by byte through index maps,
and every softmax is taken over the visible keys alone."""
from __future__ import annotations

import math

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
CODES = torch.cat([LEVELS, -LEVELS])
# byte u: five exponent bits (0: subnormal, 31: infinity or NaN) and three fraction bits
SCALES = torch.tensor([math.ldexp((u & 7) + (8 if u >> 3 else 0), max(u >> 3, 1) - 18) for u in range(248)]
                      + [math.inf] + [math.nan] * 7, dtype=torch.float64)
TOP = 0xE2


def _nearest(table: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
    """Index of the entry of the ascending table nearest to x >= 0, ties to the even index."""
    hi = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
    up, down = table[hi] - x, x - table[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x: torch.Tensor):
    """[..., D] values -> codes [..., D] (0..15) and scale bytes [..., D/16] (int64)."""
    b = x.double().cpu().unflatten(-1, (-1, 16))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], 0.0, b)
    u = _nearest(SCALES[: TOP + 1], b.abs().amax(-1) / 6)
    s = SCALES[u][..., None]
    c = _nearest(LEVELS, torch.where(s > 0, b.abs() / torch.where(s > 0, s, 1.0), 0.0))
    c = torch.where((b < 0) & (c > 0), c + 8, c)
    return torch.where(bad[..., None], 0, c).flatten(-2), torch.where(bad, 255, u)


def offsets(shape):
    """Byte offsets in a page: code byte and scale byte of (token, head, dim), K then V, [2, T, H, D]."""
    T, H, D = shape
    t, h, d = torch.arange(T)[:, None, None], torch.arange(H)[:, None], torch.arange(D)
    chunk = (t // 16 * H + h) * 18 * D
    code = [chunk + v * 9 * D + t % 16 * (D // 2) + d // 2 for v in (0, 1)]
    scale = [chunk + v * 9 * D + 8 * D + t % 16 * (D // 16) + d // 16 for v in (0, 1)]
    return torch.stack(code), torch.stack(scale)


def write(pages: torch.Tensor, shape, k, v, dest) -> None:
    """pages [P, bytes] (uint8, CPU) with the tokens k, v [n, H, D] at the token slots dest."""
    T, H, D = shape
    code_at, scale_at = offsets(shape)
    for which, x in ((0, k), (1, v)):
        c, u = quantise(x)
        for i, d in enumerate(dest.tolist()):
            if not 0 <= d < pages.shape[0] * T:
                continue
            page, t = pages[d // T], d % T
            page[code_at[which, t, :, ::2]] = (c[i][:, ::2] | c[i][:, 1::2] << 4).to(torch.uint8)
            page[scale_at[which, t, :, ::16]] = u[i].to(torch.uint8)


def read(pages: torch.Tensor, shape):
    """K and V of pages [n, bytes] in 64 bits, [n, T, H, D]."""
    code_at, scale_at = offsets(shape)
    x = pages.cpu().long()
    odd = (torch.arange(shape[2]) % 2 == 1).expand(shape)
    out = []
    for which in (0, 1):
        byte = x[:, code_at[which]]
        out.append(CODES[torch.where(odd, byte >> 4, byte & 15)] * SCALES[x[:, scale_at[which]]])
    return out


def random_pages(n: int, shape, seed: int) -> torch.Tensor:
    """n pages of random codes and scales around one (uint8, CPU)."""
    g = torch.Generator().manual_seed(seed)
    T, H, D = shape
    pages = torch.randint(0, 256, (n, T * H * D * 9 // 8), generator=g, dtype=torch.uint8)
    _, scale_at = offsets(shape)
    at = scale_at[..., ::16].reshape(-1)
    pages[:, at] = torch.randint(0x50, 0x70, (n, at.numel()), generator=g, dtype=torch.uint8)
    return pages


def attend(shape, q, pages, slots, sel, lengths, scale, cap=0.0, slopes=None, start=None, prefix=None):
    """o and lse in 64 bits, and the bound on the kernel's error in each: (o, lse, tol_o, tol_lse).

    The bound counts, to first order (5 % is added for the second):
      * the score of a key: products of halves are exact and add up in f32, at most D roundings
        of 2^-23 of the sum of magnitudes; the cap's tanh is within cap 2^-20 (a difference of
        numbers near one); the scalings, the bias and the shift by the maximum round at most
        four times, 2^-21 of the magnitudes in all (biases counted from the nearest key, which
        is how the kernel takes them). A weight moves by that relative amount, and the
        exponential adds 2^-20;
      * the weight's rounding to half for the product with V: 2^-11 relative, or 2^-25 of the
        largest weight where it is subnormal;
      * both again through the normalising sum, which adds unrounded weights (so without the
        2^-11);
      * f32 sums of the weighted values: at most n roundings of 2^-23, taken as 2^-23 of the
        magnitudes for every 16 keys of a tile and once per join;
      * the output's rounding: 2^-8 of the value for bf16, 2^-11 for fp16 (and 2^-25 where a
        half is subnormal).
    """
    B, Tq, Hq, D = q.shape
    T, H, _ = shape
    G = Hq // H
    half_step = 2.0 ** -8 if q.dtype is torch.bfloat16 else 2.0 ** -11
    o = torch.zeros((B, Tq, Hq, D), dtype=torch.float64)
    lse = torch.full((B, Tq, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    S = pages.shape[1]
    for b in range(B):
        ok = (slots[b] >= 0) & (slots[b] < S) & (sel[b] >= 0)
        if not ok.any():
            continue
        k, v = (x.flatten(0, 1) for x in read(pages[b][slots[b][ok].long()], shape))
        pos = (sel[b][ok].long()[:, None] * T + torch.arange(T)).reshape(-1)
        for t in range(Tq):
            here = int(lengths[b]) - Tq + t
            see = pos <= here
            if start is not None:
                see &= (pos >= int(start[b])) | (pos < (int(prefix[b]) if prefix is not None else 0))
            if not see.any():
                continue
            kk, vv, p = k[see], v[see], pos[see]
            for h in range(H):
                qq = q[b, t, h * G:(h + 1) * G].double()
                x = qq @ kk[:, h].T * scale
                eps = D * 2.0 ** -23 * abs(scale) * (qq.abs() @ kk[:, h].abs().T)
                if cap:
                    x = cap * torch.tanh(x / cap)
                    eps = eps + cap * 2.0 ** -20
                eps = eps + 2.0 ** -21 * x.abs()
                if slopes is not None:
                    sl = slopes[h * G:(h + 1) * G].double()[:, None]
                    x = x - sl * (here - p).double()
                    eps = eps + 2.0 ** -21 * sl.abs() * (p.max() - p).double()
                total = torch.logsumexp(x, -1)
                w = torch.exp(x - total[:, None])
                r = slice(h * G, (h + 1) * G)
                out = w @ vv[:, h]
                o[b, t, r], lse[b, t, r] = out, total
                mag = vv[:, h].abs()
                moved = (w * (eps + 2.0 ** -20)).sum(-1, keepdim=True)
                n = p.numel()
                tol = (w * (eps + 2.0 ** -20 + 2.0 ** -11 + (n / 16 + 20) * 2.0 ** -23)) @ mag + moved * out.abs()
                tol = tol + 2.0 ** -25 * mag.sum(0) + half_step * out.abs() + 2.0 ** -25
                tol_o[b, t, r] = 1.05 * tol
                tol_l[b, t, r] = 1.05 * (moved[:, 0] + 2.0 ** -21 * (total.abs() + 1))
                if slopes is not None:
                    tol_l[b, t, r] += 2.0 ** -21 * sl[:, 0].abs() * float(here - p.max())
    return o, lse, tol_o, tol_l

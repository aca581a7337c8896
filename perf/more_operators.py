"""The latent operators' cases: tokens written into latent entries (their rotary keys rotated
on the way) and read back, the two products that put latent attention into its absorbed form,
and the attention of prompts in its expanded form, in plain torch and as the framework's calls.

A token's latent is 512 values, its rotary key 64. An entry holds them in 656 bytes: 512 E4M3
codes, four fp32 scales (each for 128 codes) and the rotary key in bf16. A scale is the
smallest power of two, from 2^-126, of which 448 times is not less than the block's largest
magnitude, and a code is the one nearest to the value over it (ties to even); a block that
holds an infinity or a NaN gets a NaN for its scale.

Rotation by position p: with c_i and s_i from row p of a table (32 cosines, then 32 sines) the
pair (a, b) becomes (a c_i - b s_i, a s_i + b c_i), where pair i is dimensions 2i and 2i + 1
(interleaved) or i and i + 32 (halves).

Head h has matrices U_h and W_h of 128 x 512: a token's key is (U_h latent, rotary key), its
value W_h latent. Expanded, a query (q, r) of 128 + 64 dimensions, r rotated already, meets
those keys and values. Absorbed, the query (U_h^T q, r rotated on the way) meets the entries
themselves, and W_h is applied to what comes out.
"""
import math

import torch

own = False

LATENT, ROPE, HEAD = 512, 64, 128
BLOCK = 128  # codes to a scale
ENTRY = 656


# ------------------------------------------------------------------------------ cases
def _latents(name, B, per, dtype, pairs="interleaved", skip=0):
    """`per` tokens for each of B requests, every `skip`-th of them padding."""
    return {"name": name, "kind": "latents", "B": B, "per": per, "dtype": dtype, "pairs": pairs, "skip": skip}


def _absorbed(name, n, H, pairs="interleaved"):
    """The queries and the outputs of n tokens of H heads, before and after the attention."""
    return {"name": name, "kind": "absorbed", "n": n, "H": H, "pairs": pairs}


def _prompts(name, B, new, past, H, dtype, ragged=False, causal=True):
    """B prompts of `new` query tokens behind `past` tokens that are there already."""
    return {"name": name, "kind": "prompts", "B": B, "new": new, "past": past, "H": H, "dtype": dtype, "ragged": ragged, "causal": causal}


def listed():
    return [
        # a decode step: one new token of each of 64 requests (latency)
        _latents("latents_decode", 64, 1, "bf16"),
        # ragged prompt chunks with padding, half precision, pairs over the two halves
        _latents("latents_odd", 7, 1021, "fp16", pairs="halves", skip=13),
        # a batch of prompts stored after their prefill
        _latents("latents_prompts", 16, 8192, "bf16"),
        # one request's decode step (latency; the matrices are all there is to read)
        _absorbed("absorbed_one", 1, 128),
        # a decode step of some requests on a shard of the heads
        _absorbed("absorbed_odd", 37, 20, pairs="halves"),
        # a decode step of 64 requests, and of 256
        _absorbed("absorbed_64", 64, 128),
        _absorbed("absorbed_256", 256, 128),
        # a prompt of a line (latency)
        _prompts("prompt_short", 1, 77, 0, 16, "bf16"),
        # prompts of all lengths in one call, half precision
        _prompts("prompts_ragged", 12, 1531, 0, 16, "fp16", ragged=True),
        # a chunk of a long prompt behind the chunks before it
        _prompts("prompt_chunk", 1, 512, 15872, 64, "bf16"),
        # new tokens against a stored prefix alone, all of it seen (joined later through lse)
        _prompts("prompt_prefix", 3, 301, 4001, 32, "bf16", ragged=True, causal=False),
        # one long prompt on a shard of the heads
        _prompts("prompt_long", 1, 16384, 0, 16, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind, pairs, dtype = rng.random(), rng.choice(("interleaved", "interleaved", "halves")), rng.choice(("bf16", "bf16", "fp16"))
    if kind < 0.25:
        n = _log(rng, 1, 1 << 17)
        B = _log(rng, 1, min(256, n))
        c = _latents("", B, max(1, n // B), dtype, pairs=pairs, skip=rng.choice((0, 0, 7)))
    elif kind < 0.5:
        c = _absorbed("", _log(rng, 1, 256), rng.choice((1, 2, 5, 8, 16, 16, 20, 32, 64, 128, 128)), pairs=pairs)
    else:
        H, B = rng.choice((1, 2, 5, 8, 16, 16, 32, 64, 128)), _log(rng, 1, 16)
        keys = _log(rng, 1, 16384)
        new = _log(rng, 1, keys) if rng.random() < 0.5 else keys
        while B * H * new * keys > 16 * 16384 * 16384 or B * H * keys > 1 << 22:
            B, new, keys = max(1, B // 2), max(1, new // 2), max(1, keys * 2 // 3)
            new = min(new, keys)
        c = _prompts("", B, new, keys - new, H, dtype, ragged=rng.random() < 0.6, causal=rng.random() < 0.8)
    c.pop("name")
    return c


# ----------------------------------------------------------------------------- inputs
def _dtype(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]


def _lens(case):
    """(query tokens, key tokens) of each prompt: `new` and `past` + `new`, or spread below them."""
    got = []
    for b in range(case["B"]):
        share = 1.0 - (b * 40503 % 65536) / 65536 if case["ragged"] else 1.0
        q, past = max(1, int(case["new"] * share)), int(case["past"] * share)
        if case["ragged"] and b % 7 == 6:  # a place of the batch that has no tokens at the moment
            q, past = 0, 0
        got.append((q, past + q if case["causal"] else max(past, min(q, 1))))
    return got


def _table(rows):
    """Cosines and sines of the positions below `rows`, fp32 [rows, 64]."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def _normal(g, *shape, size=1.0):
    return torch.randn(shape, generator=g, device="cuda") * size


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "halves": case.get("pairs") == "halves"}
    if case["kind"] == "latents":
        B, per, dt = case["B"], case["per"], _dtype(case)
        n = B * per
        first = 1000 if per == 1 else 0
        size = torch.exp(0.5 * _normal(g, LATENT))  # channels of differing size, a few large ones
        size[::29] *= 6.0
        s.update(latent=(_normal(g, n, LATENT) * size).to(dt), rope=_normal(g, n, ROPE, size=2.0).to(dt))
        s["table"] = _table(first + per + 1)
        s["positions"] = (first + torch.arange(per, device="cuda", dtype=torch.int32)).repeat(B)
        place = torch.randperm(n + 3, generator=g, device="cuda")[:n]
        s["slots"] = place.to(torch.int32).view(1, n)
        dest = place.clone()
        if case["skip"]:
            dest[case["skip"] - 1:: case["skip"]] = -1
        s["dest"] = dest
        s["entries"] = torch.zeros((1, n + 3, ENTRY), dtype=torch.uint8, device="cuda")
        s["latent_out"] = torch.empty((1, n, LATENT), dtype=dt, device="cuda")
        s["rope_out"] = torch.empty((1, n, ROPE), dtype=dt, device="cuda")
        return s
    if case["kind"] == "absorbed":
        n, H, dt = case["n"], case["H"], torch.bfloat16
        s["q"] = _normal(g, n, H, HEAD + ROPE).to(dt)
        both = _normal(g, H, 2 * HEAD, LATENT, size=LATENT ** -0.5).to(dt)  # one projection, the keys' part before the values'
        s["up_k"], s["up_v"] = both[:, :HEAD], both[:, HEAD:]
        s["o"] = _normal(g, n, H, LATENT, size=0.5)
        s["positions"] = (torch.rand(n, generator=g, device="cuda") * 131072).to(torch.int32)
        s["table"] = _table(131072)
        s["q_out"] = torch.empty((n, H, LATENT + ROPE), dtype=dt, device="cuda")
        s["o_out"] = torch.empty((n, H, HEAD), dtype=dt, device="cuda")
        return s
    H, dt, lens = case["H"], _dtype(case), _lens(case)
    nq, nk = sum(q for q, _ in lens), sum(k for _, k in lens)
    starts = (lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32, device="cuda"))
    s["q"] = _normal(g, nq, H, HEAD + ROPE).to(dt)
    kv = torch.empty((nk, H, 2 * HEAD), dtype=dt, device="cuda")  # what the projection of the latents gives
    for i in range(0, nk, 4096):
        kv[i:i + 4096] = _normal(g, *kv[i:i + 4096].shape).to(dt)
    s["k"], s["v"] = kv[..., :HEAD], kv[..., HEAD:]
    s["k_rope"] = _normal(g, nk, ROPE).to(dt)
    s["q_starts"], s["k_starts"] = starts([q for q, _ in lens]), starts([k for _, k in lens])
    s["sides"] = max(q for q, _ in lens), max(k for _, k in lens)
    s["scale"] = (HEAD + ROPE) ** -0.5
    s["o"] = torch.empty((nq, H, HEAD), dtype=dt, device="cuda")
    s["lse"] = torch.empty((nq, H), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------- the plain operators
def _rotate(x, table, positions, halves):
    """x [n, ..., 64] of 16-bit floats, row i rotated by positions[i], in fp32."""
    row = table[positions.long()].view(-1, *(1,) * (x.dim() - 2), ROPE)
    c, t = row[..., :32], row[..., 32:]
    a, b = (x.float()[..., :32], x.float()[..., 32:]) if halves else (x.float()[..., 0::2], x.float()[..., 1::2])
    u, v = a * c - b * t, a * t + b * c
    return torch.cat((u, v), -1) if halves else torch.stack((u, v), -1).flatten(-2)


def _write(s, keep):
    x = s["latent"][keep].float().unflatten(-1, (-1, BLOCK))
    big = x.abs().amax(-1)
    part, power = torch.frexp(big)  # 448 is 7/8 of 2^9
    power = torch.where(big > 0, power - 9 + (part > 0.875), -126).clamp(min=-126)
    scale = torch.ldexp(torch.ones_like(big), power)
    scale = torch.where(torch.isfinite(big), scale, math.nan)
    codes = (x / scale[..., None]).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
    rope = _rotate(s["rope"][keep], s["table"], s["positions"][keep], s["halves"]).to(torch.bfloat16)
    s["entries"][0][s["dest"][keep]] = torch.cat((codes, scale.view(torch.uint8), rope.view(torch.uint8)), -1)


def _read(entries, slots, dtype):
    got = entries[0][slots[0].long()]
    codes = got[:, :LATENT].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLOCK))
    scale = got[:, LATENT:LATENT + 16].contiguous().view(torch.float32)
    rope = got[:, LATENT + 16:].contiguous().view(torch.bfloat16)
    return (codes * scale[..., None]).flatten(-2).to(dtype)[None], rope.to(dtype)[None]


def _absorb(s):
    q = torch.matmul(s["q"][..., :HEAD].float().transpose(0, 1), s["up_k"].float()).transpose(0, 1)
    r = _rotate(s["q"][..., HEAD:], s["table"], s["positions"], s["halves"])
    o = torch.matmul(s["o"].transpose(0, 1), s["up_v"].float().transpose(1, 2)).transpose(0, 1)
    return torch.cat((q, r), -1).to(torch.bfloat16), o.to(torch.bfloat16)


def _attention(s):
    c, (Lq, Lk) = s["case"], s["sides"]
    q = s["q"].float()
    iq, ik = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    q0, k0 = s["q_starts"].long(), s["k_starts"].long()
    nq, nk = q0[1:] - q0[:-1], k0[1:] - k0[:-1]
    at_q = (q0[:-1, None] + iq).clamp(max=q.shape[0] - 1)  # [B, Lq], rows behind a prompt's end among them
    at_k = (k0[:-1, None] + ik).clamp(max=s["k"].shape[0] - 1)
    seen = (ik < nk[:, None])[:, None, None, :]
    if c["causal"]:
        seen = seen & (ik <= iq[:, None] + (nk - nq)[:, None, None])[:, None]
    rope = s["k_rope"].float()[at_k][:, None].transpose(-1, -2)
    x = torch.matmul(q[at_q][..., :HEAD].transpose(1, 2), s["k"].float()[at_k].permute(0, 2, 3, 1))
    x += torch.matmul(q[at_q][..., HEAD:].transpose(1, 2), rope)
    x *= s["scale"]
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    x = torch.exp_(x.sub_(top))
    total = x.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    o = torch.matmul(x, s["v"].float()[at_k].transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    there = iq < nq[:, None]  # the prompts' own rows, in order
    return o.transpose(1, 2)[there].to(s["q"].dtype), lse.transpose(1, 2)[there]


# -------------------------------------------------------------------------------- a pass
def run(s):
    kind = s["case"]["kind"]
    if own:
        import hierarchical_kv_cache_swap_gb300 as hs
        turn = {"rotation": s["table"], "positions": s["positions"], "halves": s["halves"]} if kind != "prompts" else {}
        if kind == "latents":
            hs.write_latents(s["latent"], s["rope"], s["dest"], s["entries"][0], **turn)
            hs.read_latents(s["entries"], s["slots"], s["latent_out"], s["rope_out"])
            return s["latent_out"], s["rope_out"]
        if kind == "absorbed":
            hs.absorb_queries(s["q"], s["up_k"], s["q_out"], **turn)
            hs.expand_outputs(s["o"], s["up_v"], s["o_out"])
            return s["q_out"], s["o_out"]
        hs.attend_prompts(s["q"], s["k"], s["k_rope"], s["v"], s["q_starts"], s["k_starts"], s["o"], s["lse"], s["scale"],
                          causal=s["case"]["causal"])
        return s["o"], s["lse"]
    if kind == "latents":
        _write(s, s["dest"] >= 0)
        return _read(s["entries"], s["slots"], s["latent"].dtype)
    return _absorb(s) if kind == "absorbed" else _attention(s)


def work(case):
    if case["kind"] == "latents":
        n = case["B"] * case["per"]
        wrote = n - (n // case["skip"] if case["skip"] else 0)
        rows = case["per"] + (1000 if case["per"] == 1 else 0)
        token = 2 * (LATENT + ROPE)
        # read the tokens, write their entries; read the entries, write what they stand for
        return {"bytes": wrote * (token + ENTRY) + n * (ENTRY + token) + 16 * n + 256 * min(rows, n), "flops": 4 * n * (LATENT + ROPE)}
    H = case["H"]
    if case["kind"] == "absorbed":
        n = case["n"]
        nbytes = 4 * H * HEAD * LATENT + n * H * (2 * (HEAD + ROPE) + 2 * (LATENT + ROPE) + 4 * LATENT + 2 * HEAD) + n * 260
        return {"bytes": nbytes, "flops": 4 * n * H * HEAD * LATENT}
    pairs, nq, nk = 0, 0, 0
    for q, k in _lens(case):
        pairs += q * k - (q * (q - 1) // 2 if case["causal"] else 0)
        nq, nk = nq + q, nk + k
    nbytes = nq * H * (2 * (HEAD + ROPE) + 2 * HEAD + 4) + nk * (H * 4 * HEAD + 2 * ROPE)
    return {"bytes": nbytes, "flops": pairs * H * 2 * (HEAD + ROPE + HEAD)}


# --------------------------------------------------------------------- from the definition
def _exact_rotation(x, positions, table, halves):
    """x [n, 64] in 64 bits as pairs of complex numbers, turned."""
    i = torch.arange(32, device="cuda")
    one, two = (i, i + 32) if halves else (2 * i, 2 * i + 1)
    t = table.double()[positions.long()]
    z = torch.complex(x[:, one], x[:, two]) * torch.complex(t[:, :32], t[:, 32:])
    y = torch.empty_like(x)
    y[:, one], y[:, two] = z.real, z.imag
    return y


def _exact_codes(x):
    """What 128-value blocks of x (64 bits, finite) read back as."""
    level = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)], dtype=torch.float64,
                         device="cuda")
    powers = torch.tensor([2.0 ** e for e in range(-126, 121)], dtype=torch.float64, device="cuda")
    s = powers[torch.searchsorted(448.0 * powers, x.abs().amax(-1).contiguous())][..., None]
    y = x.abs() / s
    hi = torch.searchsorted(level, y).clamp(1, 126)
    up, down = level[hi] - y, y - level[hi - 1]
    return torch.sign(x) * level[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)] * s


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "latents":
        keep = (s["dest"] >= 0).nonzero()[:, 0]
        latent = torch.zeros((s["dest"].numel(), LATENT), dtype=torch.float64, device="cuda")
        rope = torch.zeros((s["dest"].numel(), ROPE), dtype=torch.float64, device="cuda")
        for j in keep.split(1 << 14):
            latent[j] = _exact_codes(s["latent"][j].double().view(-1, LATENT // BLOCK, BLOCK)).view(-1, LATENT)
            rope[j] = _exact_rotation(s["rope"][j].double(), s["positions"][j], s["table"], s["halves"])
        return latent[None], rope[None]
    H = case["H"]
    if case["kind"] == "absorbed":
        q, o = [], []
        for h in range(H):
            r = _exact_rotation(s["q"][:, h, HEAD:].double(), s["positions"], s["table"], s["halves"])
            q.append(torch.cat((torch.einsum("nd,dc->nc", s["q"][:, h, :HEAD].double(), s["up_k"][h].double()), r), -1))
            o.append(torch.einsum("nc,dc->nd", s["o"][:, h].double(), s["up_v"][h].double()))
        return torch.stack(q, 1), torch.stack(o, 1)
    outs = torch.zeros((s["q"].shape[0], H, HEAD), dtype=torch.float64, device="cuda")
    lses = torch.full((s["q"].shape[0], H), -math.inf, dtype=torch.float64, device="cuda")
    a, b = 0, 0
    for q, k in _lens(case):
        if q == 0:
            continue
        hidden = torch.arange(k, device="cuda") > torch.arange(q, device="cuda")[:, None] + (k - q)
        for h in range(H):
            x = s["q"][a:a + q, h].double()
            x = (x[:, :HEAD] @ s["k"][b:b + k, h].double().T + x[:, HEAD:] @ s["k_rope"][b:b + k].double().T) * s["scale"]
            if case["causal"]:
                x.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(x, -1)
            lses[a:a + q, h] = lse
            outs[a:a + q, h] = torch.exp(x - lse[:, None]) @ s["v"][b:b + k, h].double()
        a, b = a + q, b + k
    return outs, lses

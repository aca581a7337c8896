"""Refusals of the latent calls, without a GPU."""
import ctypes
import os
import re

import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs


@pytest.fixture(scope="module")
def lib():
    hs.build()
    return hs.load_library()


A = 1 << 20  # an aligned address that no accepted call reaches


def invalid(rc, message):
    assert rc == hs.HS_ERR_INVALID
    assert message in hs.last_error()


def rows(**kw):
    return hs._LatentRows(**{**dict(latent=A, rope=A, latent_stride=512, rope_stride=64), **kw})


def rotation(**kw):
    return hs._Rotation(**{**dict(table=A, rows=8, positions=A, halves=0), **kw})


def test_writes_are_checked(lib):
    def call(dtype=0, r=rows(), n=3, rot=None, dest=A, entries=A, num=4):
        return lib.hs_write_latents(None, dtype, r and ctypes.byref(r), n, rot and ctypes.byref(rot), dest, entries, num, None)
    invalid(call(dtype=2), "dtype")
    invalid(call(r=None), "null latent rows")
    invalid(call(n=-1), "negative")
    invalid(call(r=rows(latent=None)), "null latent/rope")
    invalid(call(r=rows(rope=A + 8)), "16-byte aligned")
    invalid(call(r=rows(rope_stride=63)), "16-byte aligned")
    invalid(call(num=-1), "num_entries")
    invalid(call(num=2**62), "num_entries")
    invalid(call(dest=None), "null dest")
    invalid(call(entries=None), "null dest/entries")
    invalid(call(entries=A + 4), "16-byte aligned")
    invalid(call(rot=rotation(table=None)), "without a table")
    invalid(call(rot=rotation(rows=-1)), "without a table")
    invalid(call(rot=rotation(positions=None)), "without positions")
    invalid(call(rot=rotation(table=A + 2)), "4-byte aligned")
    invalid(lib.hs_append_latents(None, None, 0, ctypes.byref(rows()), 1, None, None, A), "null context")


def test_reads_are_checked(lib):
    def call(dtype=0, entries=A, B=1, S=2, slots=A, n=3, latent=A, rope=A):
        return lib.hs_read_latents(None, dtype, entries, B, S, slots, n, latent, rope, None)
    invalid(call(dtype=-1), "dtype")
    for bad in (dict(B=-1), dict(S=-1), dict(n=-1)):
        invalid(call(**bad), "negative")
    for bad in (dict(entries=None), dict(slots=None), dict(latent=None), dict(rope=None)):
        invalid(call(**bad), "null")
    for bad in (dict(entries=A + 8), dict(latent=A + 2), dict(rope=A + 8)):
        invalid(call(**bad), "aligned")


def test_products_are_checked(lib):
    def product(**kw):
        return hs._HeadProduct(**{**dict(x=A, x_token_stride=768, x_head_stride=192, w=A, w_head_stride=65536, w_row_stride=512, out=A, n=2,
                                         heads=4), **kw})
    for call in (lambda p, rot=None: lib.hs_absorb_queries(None, p and ctypes.byref(p), rot and ctypes.byref(rot), None),
                 lambda p: lib.hs_expand_outputs(None, p and ctypes.byref(p))):
        invalid(call(None), "null product")
        invalid(call(product(n=-1)), "negative")
        for heads in (0, -1, 65536):
            invalid(call(product(heads=heads)), "heads")
        for bad in ("x", "w", "out"):
            invalid(call(product(**{bad: None})), "null")
            invalid(call(product(**{bad: A + 8})), "aligned")
        for bad in (dict(w_head_stride=0), dict(w_row_stride=-512), dict(w_row_stride=0), dict(w_head_stride=2**39)):
            invalid(call(product(**bad)), "must be positive")
        for bad in (dict(x_token_stride=770), dict(x_head_stride=2), dict(w_head_stride=4), dict(w_row_stride=516)):
            invalid(call(product(**bad)), "aligned")
    for bad in (dict(x_token_stride=0), dict(x_head_stride=-192)):
        invalid(lib.hs_absorb_queries(None, ctypes.byref(product(**bad)), None, None), "must be positive")
    assert lib.hs_absorb_queries(None, ctypes.byref(product(n=2**22 + 1)), None, None) == hs.HS_ERR_LIMIT
    invalid(lib.hs_absorb_queries(None, ctypes.byref(product()), ctypes.byref(rotation(positions=None)), None), "without positions")
    invalid(lib.hs_absorb_queries(None, ctypes.byref(product(x_token_stride=772)), None, None), "aligned")


def prompt(**kw):
    return hs._PromptAttention(**{**dict(dtype=0, B=2, heads=4, causal=1, q_rows=9, k_rows=20, q=A, q_token_stride=768, q_head_stride=192, k=A,
                                         k_token_stride=1024, k_head_stride=256, k_rope=A, k_rope_stride=64, v=A, v_token_stride=1024,
                                         v_head_stride=256, o=A, o_token_stride=512, o_head_stride=128, lse=A, q_starts=A, k_starts=A,
                                         sm_scale=0.1), **kw})


def test_prompts_are_checked(lib):
    def call(**kw):
        return lib.hs_attend_prompts(None, ctypes.byref(prompt(**kw)))
    invalid(lib.hs_attend_prompts(None, None), "null arguments")
    invalid(call(dtype=7), "dtype")
    invalid(call(B=-1), "B=-1")
    for heads in (0, 65536):
        invalid(call(heads=heads), "heads")
    for bad in (dict(q_rows=-1), dict(k_rows=-1), dict(q_rows=2**31), dict(k_rows=2**31)):
        invalid(call(**bad), "2^31")
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e31):
        invalid(call(sm_scale=scale), "sm_scale")
    for name in ("q", "o", "lse", "k", "k_rope", "v", "q_starts", "k_starts"):
        invalid(call(**{name: None}), "null")
    for name in ("q", "o", "k", "k_rope", "v"):
        invalid(call(**{name: A + 8}), "aligned")
    for name in ("q_token", "q_head", "k_token", "k_head", "k_rope", "v_token", "v_head"):
        invalid(call(**{name + "_stride": 12}), "aligned")
        for value in (0, -64, 2**39):
            invalid(call(**{name + "_stride": value}), f"{name}_stride")
    for name in ("o_token", "o_head"):
        invalid(call(**{name + "_stride": 12}), "aligned")
        invalid(call(**{name + "_stride": 0}), "overlap")
    invalid(call(o_token_stride=512, o_head_stride=120), "overlap")
    assert call(q_rows=2**31 - 256, heads=256, q_token_stride=2**20, o_token_stride=2**20) == hs.HS_ERR_LIMIT


def test_the_binding_checks_its_tensors():
    hs.build()
    lat, rope, ent = torch.zeros(3, 512, dtype=torch.bfloat16), torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(4, 656, dtype=torch.uint8)
    dest = torch.zeros(3, dtype=torch.int64)

    def refused(fn, *args, match, **kw):
        with pytest.raises((ValueError, hs.HsError), match=match):
            fn(*args, **kw)

    w = hs.write_latents
    refused(w, 3, rope, dest, ent, match="latent must be a tensor")
    refused(w, lat.float(), rope, dest, ent, match="bfloat16 or float16")
    refused(w, lat, rope.half(), dest, ent, match="one dtype")
    refused(w, lat[:, :500], rope, dest, ent, match="shape")
    refused(w, lat.t().contiguous().t(), rope, dest, ent, match="contiguous rows")
    refused(w, lat, rope, dest.int(), ent, match="dest must be")
    refused(w, lat, rope, dest, ent[:, :640], match="entries must be")
    refused(w, lat, rope, dest, ent, match="CPU")
    refused(hs.read_latents, ent.view(1, 4, 656), torch.zeros(1, 3, dtype=torch.int64), lat[None], rope[None], match="slots must be")
    refused(hs.read_latents, ent.view(1, 4, 656), torch.zeros(1, 3, dtype=torch.int32), lat[None], rope[None, :2], match="rope must be")
    q, up, out = torch.zeros(2, 4, 192, dtype=torch.bfloat16), torch.zeros(4, 128, 512, dtype=torch.bfloat16), torch.zeros(2, 4, 576, dtype=torch.bfloat16)
    refused(hs.absorb_queries, q.half(), up, out, match="q must be")
    refused(hs.absorb_queries, q, up[:3], out, match="matrices must be")
    refused(hs.absorb_queries, q, up, out[:, :, :512], match="out must be")
    refused(hs.absorb_queries, q, up, out, match="CPU")
    refused(hs.expand_outputs, torch.zeros(2, 4, 512), up, out, match="out must be")
    k, v, r = torch.zeros(5, 4, 128, dtype=torch.bfloat16), torch.zeros(5, 4, 128, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int32)
    o, lse = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 4)
    p = hs.attend_prompts
    refused(p, q, k, r, v[:4], s, s, o, lse, 0.1, match="v must have")
    refused(p, q, k.half(), r, v, s, s, o, lse, 0.1, match="k must have")
    refused(p, q, k, r[:, :32], v, s, s, o, lse, 0.1, match="k_rope")
    refused(p, q, k, r, v, s, s[:2], o, lse, 0.1, match="k_starts")
    refused(p, q, k, r, v, s[:0], s[:0], o, lse, 0.1, match="more than there are prompts")
    refused(p, q, k, r, v, s, s, o, lse.double(), 0.1, match="lse")
    refused(p, q, k, r, v, s, s, o, lse, 0.1, match="CPU")


def test_every_kernel_waits_before_it_reads_and_none_leaves_before():
    """The latent kernels are programmatic dependents: each waits, always, before its first access to
    global memory and before any way out of it."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_cache_swap_gb300", "csrc")
    found = []
    for name in ("hs_latent.cu", "hs_absorb.cu", "hs_prompt.cu"):
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__ void __launch_bounds__\([^)]*\)\s*(\w+)\s*\([^{;]*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            before, *rest = text[m.end():i].split('asm volatile("griddepcontrol.wait;" ::: "memory");')
            assert len(rest) == 1, m.group(1)
            depth = before.count("{") - before.count("}")
            assert depth == 0 and not re.search(r"\breturn\b|\bif\b|\bload\(|ld\.global|cp\.async", before), m.group(1)
            found.append(m.group(1))
    assert sorted(found) == ["absorb_kernel", "expand_few_kernel", "expand_many_kernel", "prompt_kernel", "read_kernel", "write_kernel"]


def test_the_most_tokens_absorbed_are_what_a_grid_holds(lib):
    """65535 tiles of 64 tokens: one more is refused, not left to the launch to fail."""
    for n in (65535 * 64 + 1, 2**22):
        p = hs._HeadProduct(x=A, x_token_stride=192, x_head_stride=192, w=A, w_head_stride=128 * 512, w_row_stride=512, out=A, n=n, heads=1)
        assert lib.hs_absorb_queries(None, ctypes.byref(p), None, None) == hs.HS_ERR_LIMIT


def body(name, kernel):
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_cache_swap_gb300", "csrc")
    with open(os.path.join(csrc, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    i = start = text.index("{", re.search(r"__global__ void __launch_bounds__\([^)]*\)\s*" + kernel + r"\b", text).end())
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[start:i]


def test_no_warp_leaves_a_loop_whose_barriers_the_others_wait_at():
    """Warps may differ in whether a wait ran out: none of them leaves the output expansion's loop, which
    holds barriers of the group."""
    loop = body("hs_absorb.cu", "expand_many_kernel").split("for (int k = 0; t0 < p.n;")[1]
    assert loop.count("bar.sync") == 2
    assert not re.search(r"\b(break|return|continue|goto)\b", loop)


def test_the_softmax_warps_meet_again_before_their_stores_are_waited_for():
    """Threads differ in how many values behind a prompt's end they make zeros, and the wait for a
    warp's stores to tensor memory is the whole warp's."""
    zeroes = body("hs_prompt.cu", "prompt_kernel").split("if (live < 64)")[1]
    assert zeroes.index("fence_async_smem();") < zeroes.index("__syncwarp();") < zeroes.index("tmem_wait_st();")

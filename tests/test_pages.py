"""4-bit pages without a GPU: the format's model against itself, the calls' refusals."""
import ctypes
import math

import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import page_models as pm


@pytest.fixture(scope="module")
def lib():
    hs.build()
    return hs.load_library()


def test_scale_table_is_the_half_precision_prefix():
    u = torch.arange(248, dtype=torch.int16)
    assert torch.equal((u << 7).view(torch.float16).double(), pm.SCALES[:248])
    assert pm.SCALES[pm.TOP] == 10240 and 6 * pm.SCALES[pm.TOP] <= 65504


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_model_rounds_to_the_nearest_code_and_reads_back_exactly(dtype):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn((64, 32), generator=g) * torch.exp(2 * torch.randn((64, 1), generator=g))).to(dtype)
    c, u = pm.quantise(x)
    y = (pm.CODES[c].unflatten(-1, (-1, 16)) * pm.SCALES[u][..., None]).flatten(-2)
    assert torch.equal(y.to(dtype).double(), y)  # six significant bits
    s = pm.SCALES[u].repeat_interleave(16, -1)
    err = (x.double() - y).abs()
    other = (x.double()[..., None] - pm.CODES * s[..., None]).abs().amin(-1)
    assert torch.equal(err, other)  # no other code of that scale is nearer
    a = x.double().unflatten(-1, (-1, 16)).abs().amax(-1) / 6
    assert torch.equal((pm.SCALES[u] - a).abs(), (pm.SCALES[: pm.TOP + 1] - a[..., None]).abs().amin(-1))


def test_model_writes_and_reads_pages():
    shape = (32, 3, 64)
    pages = pm.random_pages(4, shape, 0)
    before = pages.clone()
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn((3, 3, 64), generator=g), torch.randn((3, 3, 64), generator=g)
    pm.write(pages, shape, k, v, torch.tensor([5, 95, -1]))
    kr, vr = pm.read(pages, shape)
    for x, y in ((k, kr), (v, vr)):
        c, u = pm.quantise(x)
        want = (pm.CODES[c].unflatten(-1, (-1, 16)) * pm.SCALES[u][..., None]).flatten(-2)
        assert torch.equal(y[0, 5], want[0]) and torch.equal(y[2, 31], want[1])
    same = pages == before
    assert same[1].all() and same[3].all()
    assert int((~same).sum()) <= 2 * 2 * 3 * 64 * 9 // 16


def test_model_attention_agrees_with_library_functions():
    shape = (16, 2, 64)
    pages = pm.random_pages(3, shape, 5).view(1, 3, -1)
    q = torch.randn((1, 1, 4, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    slots, sel = torch.tensor([[2, 0]]), torch.tensor([[0, 1]])
    o, lse, _, _ = pm.attend(shape, q, pages, slots, sel, torch.tensor([27]), 0.125)
    k, v = (x[[2, 0]].flatten(0, 1)[:27].repeat_interleave(2, 1).transpose(0, 1) for x in pm.read(pages[0], shape))
    want = torch.nn.functional.scaled_dot_product_attention(q[0, 0][:, None].double(), k, v, scale=0.125)
    assert (o[0, 0] - want[:, 0]).abs().max() < 1e-12
    assert (lse[0, 0] - torch.logsumexp((k @ q[0, 0].double()[..., None])[..., 0] * 0.125, -1)).abs().max() < 1e-12


@pytest.mark.parametrize("shape,n", [((16, 8, 128), 18432), ((256, 1, 64), 18432), ((48, 3, 256), 41472),
                                     ((0, 8, 128), 0), ((24, 8, 128), 0), ((272, 8, 128), 0), ((16, 0, 128), 0),
                                     ((16, 8, 96), 0), ((256, 65535, 256), 0), ((-16, 8, 128), 0)])
def test_page_bytes(lib, shape, n):
    assert lib.hs_page_bytes(ctypes.byref(hs._PageShape(*shape))) == n
    if n:
        assert hs.PageShape(*shape).bytes == n
    else:
        with pytest.raises(ValueError):
            hs.PageShape(*shape).bytes
    assert lib.hs_page_bytes(None) == 0


GOOD = hs._PageShape(16, 8, 128)


def _ref(x):
    return ctypes.byref(x)


@pytest.mark.parametrize("what,shape,dtype,rows,n,dest,pages,P", [
    ("null page shape", None, 0, (32, 32, 1024, 128, 1024, 128), 4, 8, 16, 1),
    ("unsupported", hs._PageShape(24, 8, 128), 0, (32, 32, 1024, 128, 1024, 128), 4, 8, 16, 1),
    ("dtype", GOOD, 2, (32, 32, 1024, 128, 1024, 128), 4, 8, 16, 1),
    ("null token rows", GOOD, 0, None, 4, 8, 16, 1),
    ("negative", GOOD, 0, (32, 32, 1024, 128, 1024, 128), -1, 8, 16, 1),
    ("null k", GOOD, 0, (0, 32, 1024, 128, 1024, 128), 4, 8, 16, 1),
    ("aligned", GOOD, 0, (34, 32, 1024, 128, 1024, 128), 4, 8, 16, 1),
    ("aligned", GOOD, 0, (32, 32, 1024, 132, 1024, 128), 4, 8, 16, 1),
    ("null dest", GOOD, 0, (32, 32, 1024, 128, 1024, 128), 4, 0, 16, 1),
    ("null dest", GOOD, 0, (32, 32, 1024, 128, 1024, 128), 4, 8, 0, 1),
    ("aligned", GOOD, 0, (32, 32, 1024, 128, 1024, 128), 4, 8, 24, 1),
    ("num_pages", GOOD, 0, (32, 32, 1024, 128, 1024, 128), 4, 8, 16, -1),
    ("num_pages", GOOD, 0, (32, 32, 1024, 128, 1024, 128), 4, 8, 16, 2**62),
])
def test_write_tokens_refuses_before_touching_cuda(lib, what, shape, dtype, rows, n, dest, pages, P):
    rows = None if rows is None else _ref(hs._TokenRows(*rows))
    assert lib.hs_write_tokens(None, None if shape is None else _ref(shape), dtype, rows, n, dest, pages, P,
                               None) == hs.HS_ERR_INVALID
    assert what in hs.last_error()


def test_append_tokens_refuses_a_null_context(lib):
    assert lib.hs_append_tokens(None, None, _ref(GOOD), 0, _ref(hs._TokenRows(16, 16, 8, 8, 8, 8)), 1, None,
                                4) == hs.HS_ERR_INVALID
    assert lib.hs_status_word(None) is None


@pytest.mark.parametrize("what,args", [
    ("unsupported", (hs._PageShape(16, 8, 80), 0, 16, 1, 1, 4, 1, 16, 16)),
    ("dtype", (GOOD, -1, 16, 1, 1, 4, 1, 16, 16)),
    ("negative", (GOOD, 0, 16, -1, 1, 4, 1, 16, 16)),
    ("negative", (GOOD, 0, 16, 1, 1, 4, -1, 16, 16)),
    ("null", (GOOD, 0, 0, 1, 1, 4, 1, 16, 16)),
    ("null", (GOOD, 0, 16, 1, 1, 0, 1, 16, 16)),
    ("null", (GOOD, 0, 16, 1, 1, 4, 1, 0, 16)),
    ("aligned", (GOOD, 0, 16, 1, 1, 4, 1, 16, 18)),
])
def test_read_pages_refuses_before_touching_cuda(lib, what, args):
    shape, dtype, pages, B, S, slots, n, k, v = args
    assert lib.hs_read_pages(None, _ref(shape), dtype, pages, B, S, slots, n, k, v, None) == hs.HS_ERR_INVALID
    assert what in hs.last_error()


def _attention(**change):
    a = dict(shape=GOOD, dtype=0, B=1, S=4, k=2, q_heads=16, q_tokens=1, q=16, q_batch_stride=2048, q_token_stride=2048,
             q_head_stride=128, o=16, o_batch_stride=2048, o_token_stride=2048, o_head_stride=128, lse=4, pages=16,
             slots=4, selections=4, lengths=4, sm_scale=0.1, softcap=0.0, slopes=None, start=None, prefix=None,
             status=None)
    a.update(change)
    return hs._PageAttention(**a)


@pytest.mark.parametrize("what,change,code", [
    ("unsupported", {"shape": hs._PageShape(16, 8, 32)}, hs.HS_ERR_INVALID),
    ("dtype", {"dtype": 7}, hs.HS_ERR_INVALID),
    ("negative", {"k": -1}, hs.HS_ERR_INVALID),
    ("negative", {"B": -1}, hs.HS_ERR_INVALID),
    ("q_heads", {"q_heads": 12}, hs.HS_ERR_INVALID),
    ("q_heads", {"q_heads": 0}, hs.HS_ERR_INVALID),
    ("q_tokens", {"q_tokens": 0}, hs.HS_ERR_INVALID),
    ("2^20", {"q_tokens": 1 << 17}, hs.HS_ERR_LIMIT),
    ("2^30", {"S": (1 << 30) + 1}, hs.HS_ERR_LIMIT),
    ("2^30", {"k": (1 << 30) + 1}, hs.HS_ERR_LIMIT),
    ("sm_scale", {"sm_scale": math.inf}, hs.HS_ERR_INVALID),
    ("sm_scale", {"sm_scale": math.nan}, hs.HS_ERR_INVALID),
    ("softcap", {"softcap": -1.0}, hs.HS_ERR_INVALID),
    ("softcap", {"softcap": math.nan}, hs.HS_ERR_INVALID),
    ("null q", {"q": None}, hs.HS_ERR_INVALID),
    ("null q", {"lengths": None}, hs.HS_ERR_INVALID),
    ("null pages", {"slots": None}, hs.HS_ERR_INVALID),
    ("null pages", {"pages": None}, hs.HS_ERR_INVALID),
    ("aligned", {"q": 24}, hs.HS_ERR_INVALID),
    ("aligned", {"o_head_stride": 4}, hs.HS_ERR_INVALID),
    ("overlap", {"o_head_stride": 0}, hs.HS_ERR_INVALID),
    ("overlap", {"o_head_stride": -120}, hs.HS_ERR_INVALID),
    ("overlap", {"q_tokens": 2, "o_token_stride": 64}, hs.HS_ERR_INVALID),
    ("overlap", {"B": 2, "o_batch_stride": 0}, hs.HS_ERR_INVALID),
])
def test_attend_pages_refuses_before_touching_cuda(lib, what, change, code):
    assert lib.hs_attend_pages(None, _ref(_attention(**change))) == code
    assert what in hs.last_error()
    assert lib.hs_attend_pages(None, None) == hs.HS_ERR_INVALID


def test_binding_checks_shapes_and_types_before_any_call():
    shape = (16, 2, 64)
    E = 16 * 2 * 64 * 9 // 8
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    dest, pages = torch.zeros(3, dtype=torch.int64), torch.zeros((4, E), dtype=torch.uint8)
    for args in [(k[:, :1], k, dest, pages), (k, k.half(), dest, pages), (k, k, dest.int(), pages),
                 (k, k, dest[:2], pages), (k, k, dest, pages[:, :-16]), (k.transpose(1, 2), k, dest, pages)]:
        with pytest.raises(ValueError):
            hs.write_tokens(shape, *args)
    slots = torch.zeros((2, 3), dtype=torch.int32)
    p3, out = pages.view(2, 2, E), torch.zeros((2, 48, 2, 64), dtype=torch.bfloat16)
    for args in [(p3[:, :, ::2], slots, out, out), (p3, slots.long(), out, out), (p3, slots, out[:, :32], out),
                 (p3[:1], slots, out, out), (p3, slots, out, out.half())]:
        with pytest.raises(ValueError):
            hs.read_pages(shape, *args)
    q, lse = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 1, 4))
    lengths = torch.zeros(2, dtype=torch.int32)
    good = dict(q=q, pages=p3, slots=slots, selections=slots, lengths=lengths, o=q.clone(), lse=lse)
    for change in [dict(q=q.half()), dict(o=q[:, :, :2]), dict(lse=lse.double()), dict(lse=lse[:, :, :2]),
                   dict(selections=slots[:, :2]), dict(lengths=lengths.long()), dict(slopes=torch.zeros(3)),
                   dict(start=torch.zeros(2)), dict(prefix=lengths[:1]), dict(pages=pages.view(4, 1, E)),
                   dict(q=torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16))]:
        with pytest.raises(ValueError):
            hs.attend_pages(shape, sm_scale=0.1, **{**good, **change})

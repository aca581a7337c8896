"""The waits within the latent kernels run out in bounded time, report it and leave the GPU usable: with
stalled waits a kernel's first copy is announced and never made, so that the roles that wait for it,
and those that wait for them, give up."""
import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import latent_models as lm
from tests.test_gpu_latents import gen, normal, prompts, status_word
from tests.test_gpu_timeout import LIMIT_NS, gpu_ms

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


@pytest.fixture
def stalled():
    """Calls `fn` with waits of 1 ms that run out; ms on the GPU."""
    def call(fn):
        hs.set_latent_waits(LIMIT_NS, stall=True)
        try:
            return gpu_ms(fn)
        finally:
            hs.set_latent_waits()
    yield call
    hs.set_latent_waits()


def in_time(ms):
    assert 0.5 <= ms <= 50.0, f"a stalled call took {ms:.3f} ms on the GPU with a 1 ms limit of a wait"


def test_prompts(stalled):
    lens, H = [(200, 300), (1, 128), (140, 90)], 3
    q, k, r, v, qs, ks = prompts(lens, H, BF16, 5)
    o, lse = torch.full((341, H, 128), 7.0, dtype=BF16, device="cuda"), torch.full((341, H), 7.0, device="cuda")
    word = status_word()

    def call():
        hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, status=word)

    in_time(stalled(call))
    assert int(word) == hs.HS_STATUS_TIMEOUT
    assert (torch.isnan(o) | (o == 7)).all() and (torch.isnan(lse) | (lse == 7)).all()
    assert torch.isnan(o[:200]).any()
    word.zero_()
    call()
    assert int(word) == 0
    a, c = 0, 0
    for lq, lk in lens:
        wo, wl, bo, bl = lm.attend(q[a:a + lq], k[c:c + lk], r[c:c + lk], v[c:c + lk], 0.1, True, BF16)
        assert lm.near(o[a:a + lq], wo, bo) and lm.near(lse[a:a + lq], wl, bl)
        a, c = a + lq, c + lk


@pytest.fixture
def short():
    hs.set_latent_waits(10 * LIMIT_NS)
    yield
    hs.set_latent_waits()


def test_a_prompt_that_takes_longer_than_the_limit_of_a_wait(short):
    """The look-up waits for as long as an item's keys take: that is not a hand-off lost.

    Values of 1 give 1: the f32 sums of 2^23 keys, 16 at a time (the products, each addition truncated)
    and 128 at a time (the weights), are off by 2^19 2^-23 and 2^16 2^-24 at most, the result by 2^-8."""
    n = 1 << 23
    q, k, r = normal(gen(1), 3, 1, 192).to(BF16), torch.empty((n, 1, 128), dtype=BF16, device="cuda"), torch.zeros((n, 64), dtype=BF16, device="cuda")
    for i in range(0, n, n // 8):
        k[i:i + n // 8] = normal(gen(i + 2), n // 8, 1, 128).to(BF16)
    v = torch.ones_like(k)
    qs, ks = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"), torch.tensor([0, n, n], dtype=torch.int32, device="cuda")
    o, lse, word = torch.empty((3, 1, 128), dtype=BF16, device="cuda"), torch.empty((3, 1), device="cuda"), status_word()
    ms = gpu_ms(lambda: hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, causal=False, status=word))
    assert ms > 12, "the item has to last for longer than the limit"
    assert int(word) == 0
    assert ((o[0].double() - 1).abs() <= 2.0 ** -4 + 2.0 ** -7).all() and not o[1:].any()
    x = torch.cat([(c[:, 0].double() @ q[0, 0, :128].double()) * 0.1 for c in k.split(n // 8)])
    assert abs(float(lse[0]) - float(torch.logsumexp(x, 0))) <= 2.0 ** -8 + 2.0 ** -12
    assert torch.isinf(lse[1:]).all()


@pytest.mark.parametrize("B,H", [(1 << 21, 1), (1 << 17, 64)])
def test_a_search_that_takes_longer_than_the_limit_of_a_wait(short, B, H):
    """Two prompts with rows, the first and the last of very many: the others have none."""
    q, k, r, v, *_ = prompts([(40, 40), (30, 50)], H, BF16, 8)
    qs, ks = (torch.full((B + 1,), a, dtype=torch.int32, device="cuda") for a in (40, 40))
    qs[0], ks[0], qs[-1], ks[-1] = 0, 0, 70, 90
    o, lse, word = torch.empty((70, H, 128), dtype=BF16, device="cuda"), torch.empty((70, H), device="cuda"), status_word()
    ms = gpu_ms(lambda: hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, status=word))
    assert ms > 12, "the search has to last for longer than the limit"
    assert int(word) == 0
    for a, b, c, d in ((0, 40, 0, 40), (40, 70, 40, 90)):
        wo, wl, bo, bl = lm.attend(q[a:b], k[c:d], r[c:d], v[c:d], 0.1, True, BF16)
        assert lm.near(o[a:b], wo, bo) and lm.near(lse[a:b], wl, bl)


@pytest.mark.parametrize("n,H", [(5, 2), (100, 40)])
def test_absorbed_queries(stalled, n, H):
    """Rows are NaN but for their rotary values, and nothing behind them is written."""
    q, up = normal(gen(1), n, H, 192).to(BF16), normal(gen(2), H, 128, 512).to(BF16)
    out = torch.full((n + 70, H, 576), 7.0, dtype=BF16, device="cuda")
    word = status_word()
    in_time(stalled(lambda: hs.absorb_queries(q, up, out[:n], status=word)))
    assert int(word) == hs.HS_STATUS_TIMEOUT
    assert torch.isnan(out[:n, :, :512]).all() and torch.equal(out[:n, :, 512:], q[..., 128:]) and (out[n:] == 7).all()
    word.zero_()
    hs.absorb_queries(q, up, out[:n], status=word)
    ref = torch.einsum("nhd,hdc->nhc", q[..., :128].double(), up.double())
    size = torch.einsum("nhd,hdc->nhc", q[..., :128].double().abs(), up.double().abs())
    assert ((out[:n, :, :512].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 130 * 2.0 ** -23 * size).all()
    assert int(word) == 0 and (out[n:] == 7).all()


@pytest.mark.parametrize("n,H", [(200, 40), (900, 152)])
def test_expanded_outputs(stalled, n, H):
    o, up = normal(gen(1), n, H, 512), normal(gen(2), H, 128, 512).to(BF16)
    out = torch.full((n + 70, H, 128), 7.0, dtype=BF16, device="cuda")
    word = status_word()
    in_time(stalled(lambda: hs.expand_outputs(o, up, out[:n], status=word)))
    assert int(word) == hs.HS_STATUS_TIMEOUT
    assert torch.isnan(out[:n]).all() and (out[n:] == 7).all()
    in_time(stalled(lambda: hs.expand_outputs(o, up, out[:n])))
    word.zero_()
    hs.expand_outputs(o, up, out[:n], status=word)
    assert int(word) == 0
    ref = torch.einsum("nhc,hec->nhe", o.double(), up.double())
    size = torch.einsum("nhc,hec->nhe", o.double().abs(), up.double().abs())
    assert ((out[:n].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 514 * 2.0 ** -23) * size).all()
    assert (out[n:] == 7).all()
    for bad in (word.cpu(), status_word().long(), torch.zeros(2, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError, match="status must be"):
            hs.expand_outputs(o, up, out[:n], status=bad)


def test_a_limit_that_ordinary_waits_do_not_keep():
    """1 us: waits run out anywhere, with copies and products under way; each row is then right or NaN or, of a
    prompt, as it was, what is not right is reported, and the next calls are as ever."""
    H, lens = 24, [(300, 700), (33, 33), (129, 1400)] * 4
    q, k, r, v, qs, ks = prompts(lens, H, BF16, 6)
    m, n = q.shape[0], 300
    x, w, s = normal(gen(1), n, H, 192).to(BF16), normal(gen(2), H, 256, 512).to(BF16), normal(gen(3), n, H, 512)

    def calls():
        words = [status_word() for _ in range(3)]
        o, lse = torch.full((m, H, 128), 7.0, dtype=BF16, device="cuda"), torch.full((m, H), 7.0, device="cuda")
        qo, oo = torch.zeros((n, H, 576), dtype=BF16, device="cuda"), torch.zeros((n, H, 128), dtype=BF16, device="cuda")
        hs.attend_prompts(q, k, r, v, qs, ks, o, lse, 0.1, status=words[0])
        hs.absorb_queries(x, w[:, :128], qo, status=words[1])
        hs.expand_outputs(s, w[:, 128:], oo, status=words[2])
        torch.cuda.synchronize()
        return (o, lse, qo, oo), [int(a) for a in words]

    want, words = calls()
    assert words == [0, 0, 0]
    hs.set_latent_waits(1000)
    try:
        for _ in range(4):
            got, words = calls()
            assert all(a in (0, hs.HS_STATUS_TIMEOUT) for a in words)
            for i, word in ((0, words[0]), (1, words[0]), (2, words[1]), (3, words[2])):
                same = (got[i] == want[i]) | torch.isnan(got[i]) | ((got[i] == 7) if i < 2 else False)
                assert same.all() and (word or torch.equal(got[i], want[i]))
    finally:
        hs.set_latent_waits()
    got, words = calls()
    assert words == [0, 0, 0] and all(torch.equal(a, b) for a, b in zip(got, want))

"""Page calls directly behind a resolution of more requests than SMs: its chunks' fetches have all
ended when the page calls begin, whichever of them takes longest."""
import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs
from tests import page_models as pm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B", [320, 470])
def test_tokens_appended_to_pages_whose_fetch_has_just_been_enqueued(B, captured):
    """Only the first requests miss, so the later chunks' fetches have nothing to copy. Tokens join
    the pages being fetched: neither place may be left with the bytes from before."""
    shape, C, k = (16, 4, 128), 20, 16
    E = hs.PageShape(*shape).bytes
    ctx = hs.Context(B, C, k, E)
    before = pm.random_pages(C, shape, 3)
    busy = B // 4
    sel = torch.full((B, k), -1, dtype=torch.int32)
    sel[:busy] = torch.arange(k, dtype=torch.int32) + 2
    at = torch.full((B,), -1, dtype=torch.int32)
    at[:busy] = (torch.arange(busy) * 7 % k + 2) * 16 + torch.arange(busy) % 16
    kv = torch.randn((2, B, 4, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    sel_d, at_d, kv_d = sel.cuda(), at.cuda(), kv.cuda()
    out, miss = torch.full_like(sel_d, -1), torch.empty(B, dtype=torch.int32, device="cuda")
    ko = torch.empty((B, k * 16, 4, 128), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)

    def step():
        ctx.resolve(sel_d, out, miss)
        ctx.append_tokens(shape, kv_d[0], kv_d[1], at_d)
        ctx.read_pages(shape, out, ko, vo)

    if captured:
        ctx.read_pages(shape, out, ko, vo)  # loads the kernel
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            step()
        step = graph.replay
    for _ in range(3):
        ctx.host_kv()[..., :E] = before.numpy()
        ctx.reset()
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        assert ctx.status() == 0 and int(miss.sum()) == busy * k
        want = before.expand(B, C, E).clone()
        pm.write(want.view(B * C, E), shape, kv[0, :busy], kv[1, :busy], torch.arange(busy) * C * 16 + at[:busy].long())
        host = torch.from_numpy(ctx.host_kv()[..., :E].copy())
        assert torch.equal(host, want)
        slots = out[:busy].long().cpu()
        rows = torch.arange(busy)[:, None]
        assert torch.equal(ctx.device_kv().view(B, k, E).cpu()[rows, slots], want[rows, sel[:busy].long()])
        b = busy - 1
        assert torch.equal(ko[b].cpu().double().view(k, 16, 4, 128), pm.read(want[b, 2:2 + k], shape)[0])
    ctx.close()

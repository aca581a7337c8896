"""The compiled binding of the page calls with tensors that have no memory."""
import pytest
import torch

import hierarchical_kv_cache_swap_gb300 as hs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    hs.build()


def test_tensors_without_memory_are_an_error():
    """Fake tensors have a device and a shape but no pointer: an ordinary error, at every call."""
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    shape = (16, 2, 64)
    E = hs.PageShape(*shape).bytes
    ctx = hs.Context(1, 4, 2, E)
    with fake.FakeTensorMode():
        empty = lambda *size, dtype: torch.empty(size, dtype=dtype, device="cuda")
        i32 = lambda *size: empty(*size, dtype=torch.int32)
        bf16 = lambda *size: empty(*size, dtype=torch.bfloat16)
        k, slots, out, q = bf16(1, 2, 64), i32(1, 2), bf16(1, 32, 2, 64), bf16(1, 1, 2, 64)
        calls = [
            lambda: ctx.read_pages(shape, slots, out, out),
            lambda: ctx.append_tokens(shape, k, k, i32(1)),
            lambda: ctx.attend_pages(shape, q, slots, slots, i32(1), q, empty(1, 1, 2, dtype=torch.float32), 0.1),
            lambda: hs.write_tokens(shape, k, k, empty(1, dtype=torch.int64), empty(3, E, dtype=torch.uint8)),
            lambda: hs.read_pages(shape, empty(1, 3, E, dtype=torch.uint8), slots, out, out),
        ]
        for call in calls:
            for _ in range(2):
                with pytest.raises((RuntimeError, ValueError)):  # hs.HsError is a RuntimeError
                    call()
    # and the calls go on working
    slots = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    out = torch.ones((1, 32, 2, 64), dtype=torch.bfloat16, device="cuda")
    ctx.read_pages(shape, slots, out, out.clone())
    assert not out.any()
    ctx.close()

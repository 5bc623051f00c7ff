"""The batch after an eviction (EvictPlan.indices, freed), whatever becomes of the
caller's page table."""
import pytest
import torch

from tests.test_evict import Cache
from tests.test_prefill import BF16


def pages_after(c, keep):
    """The page ids that stay and those that are freed, in the table's order."""
    stay, free = [], []
    for i, length in enumerate(c.lengths):
        ids = c.ids[c.indptr[i]:c.indptr[i + 1]].tolist()
        n = -(-min(int(length), keep) // 16)
        stay += ids[:n]
        free += ids[n:]
    return stay, free


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["device", "host"])
@pytest.mark.parametrize("on_stream", [False, True])
def test_pages_after_the_table_was_rewritten(lib, cuda, where, on_stream):
    """The order of calls that a serving loop has: the table is overwritten with what
    stays, then the freed pages go back to the pool."""
    c = Cache([100, 0, 64, 17, 300], 2, 64, BF16)
    if where == "host":
        c.indices = torch.from_numpy(c.ids.copy()).pin_memory()
    table = c.indices
    kw = {"stream": torch.cuda.Stream()} if on_stream else {}
    torch.cuda.synchronize()
    p = c.plan(lib, 32, **kw)
    torch.cuda.synchronize()
    stay, free = pages_after(c, 32)
    new = p.indices
    table[:len(new)].copy_(new)
    table[len(new):] = 0
    assert p.indices.tolist() == stay and p.freed.tolist() == free
    assert p.indices.dtype == p.freed.dtype == torch.int32
    assert p.indices.is_cuda == (where == "device") == p.freed.is_cuda
    lib.plan(p.indptr, p.indices, p.last_page_len, 2, 2, 64, 16)


@pytest.mark.gpu
def test_pages_are_read_on_the_plan_stream(lib, cuda):
    """A table that a stream's earlier work writes, planned on that stream."""
    c = Cache([4000], 2, 64, BF16, seed=3)
    right, side = c.indices.clone(), torch.cuda.Stream()
    a = torch.randn(4096, 4096, device=cuda)
    c.indices.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):  # some ms of work in front of the write
            a = (a @ a).clamp_(-1, 1)
        c.indices.copy_(right)
    p = c.plan(lib, 100, stream=side)
    after = p.indices, p.freed
    torch.cuda.synchronize()
    stay, free = pages_after(c, 100)
    assert after[0].tolist() == stay and after[1].tolist() == free

"""check() reads and clears the device-check word on the stream it is given: it
does not wait for the default stream, nor leave the clear to it (where it could
come after what a kernel on another stream sets next)."""
import numpy as np
import pytest
import torch

from tests.test_append import BF16, E4M3, Batch

pytestmark = pytest.mark.gpu
SHAPE = (8, 2, 128, 16)


def append_plan(lib, cuda):
    b = Batch([0, 0], [20, 3], 8, 2, 128, BF16, BF16)
    b.indices[1] = b.num_pages
    p = b.plan(lib)
    return p, lambda s: p.run(b.k, b.v, b.kv, stream=s), p.check


def decode_plan(lib, cuda):
    ids = torch.tensor([0, 9, 1], dtype=torch.int32, device=cuda)
    kv = torch.zeros((3, 2, 16, 2, 128), dtype=BF16, device=cuda)
    q = torch.zeros((2, 8, 128), dtype=BF16, device=cuda)
    p = lib.plan([0, 2, 3], ids, [16, 3], *SHAPE)
    o, lse = torch.empty_like(q), torch.empty((2, 8), device=cuda)
    return p, lambda s: p.run(q, kv, out=o, lse=lse, stream=s), p.check


def cascade_plan(lib, cuda):
    pre = torch.tensor([0, 9], dtype=torch.int32, device=cuda)
    own = torch.tensor([1, 2], dtype=torch.int32, device=cuda)
    kv = torch.zeros((3, 2, 16, 2, 128), dtype=BF16, device=cuda)
    q = torch.zeros((2, 8, 128), dtype=BF16, device=cuda)
    p = lib.cascade_plan(pre, np.array([0, 1, 2]), own, [16, 3], *SHAPE)
    o, lse = torch.empty_like(q), torch.empty((2, 8), device=cuda)
    return p, lambda s: p.run(q, kv, out=o, lse=lse, stream=s), p.check


def unified_max_plan(lib, cuda):
    ids = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda)
    kv = torch.ones((3, 2, 16, 2, 128), dtype=BF16, device=cuda)
    q = torch.full((2, 8, 128), 8.0, dtype=BF16, device=cuda)
    p = lib.plan([0, 2, 3], ids, [16, 3], *SHAPE)
    o, lse = torch.empty_like(q), torch.empty((2, 8), device=cuda)
    return (p, lambda s: p.run_unified_max(q, kv, -1000.0, out=o, lse=lse, stream=s),
            lambda s: int(p.unified_max_fallbacks(s) > 0))


@pytest.mark.parametrize("make", [append_plan, decode_plan, cascade_plan, unified_max_plan])
def test_check_does_not_use_the_default_stream(lib, cuda, make):
    p, run, check = make(lib, cuda)
    side = torch.cuda.Stream()
    run(side)
    assert check(side) & 1 == 1 and check(side) == 0      # loads what it needs
    torch.cuda.synchronize()
    run(side)
    torch.cuda._sleep(400_000_000)                          # 0.2 s of the default stream
    assert check(side) & 1 == 1
    assert not torch.cuda.default_stream().query()
    run(side)
    assert check(side) & 1 == 1 and check(side) == 0
    assert not torch.cuda.default_stream().query()
    torch.cuda.synchronize()

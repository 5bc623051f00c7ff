"""Evictions that follow each other, and scales moved by clusters of CTAs."""
import numpy as np
import pytest
import torch

from tests.test_evict import Cache
from tests.test_prefill import BF16, E4M3


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hkv,keep,recent", [([700, 50, 400], 3, 96, 16), ([20000], 1, 3000, 33)])
def test_one_plan_run_again(lib, cuda, lengths, hkv, keep, recent):
    """New weights over the same slots, then the same plan: each run is the definition on
    what it finds."""
    c = Cache(lengths, hkv, 64, BF16, seed=8)
    p = c.plan(lib, keep, recent)
    for turn in range(3):
        want = c.expected(keep, recent)
        c.run(p)
        assert p.check() == 0
        assert all(np.array_equal(x, y) for x, y in zip(c.state(), want))
        if turn == 1:
            g = torch.Generator(device="cuda").manual_seed(9)
            c.w.copy_(torch.rand(c.w.shape, generator=g, device=cuda))


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hkv,keep,recent", [
    ([2500], 1, 700, 10), ([5000, 300], 2, 2100, 0), ([20000], 2, 8000, 33), ([20000] * 12, 8, 900, 9)])
def test_token_scales_move_with_their_tokens(lib, cuda, lengths, hkv, keep, recent):
    """Clusters of two to eight CTAs, and of one."""
    Cache(lengths, hkv, 128, E4M3, seed=4, token_scales=True).check(lib, keep, recent)

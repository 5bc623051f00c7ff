"""Prompt attention whose repair of rows takes longer than the bound on the kernel's
waits (2 s): the CTA's other warps, and its next items, wait for it.  Bounds as in
test_prefill.py."""
import numpy as np
import pytest
import torch

from tests.test_prefill import BF16, Batch


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [20005, 200005])
def test_rows_that_are_computed_again_over_long_contexts(lib, cuda, ctx):
    """V of the last token is not finite, in one head: 127 rows of a block walk all
    tokens they see, 32 a warp, several seconds at the longer context.  Two items a CTA,
    all with ragged ends; that item is one of the first, so that its CTA's next one
    comes behind it."""
    hkv, n = 8, 38 * 256  # 304 items for 152 CTAs
    b = Batch([ctx], [n], hkv, hkv, 64, BF16, seed=40)
    offsets, items, merge, slots = lib.plan_prefill_host(b.indptr, b.last, b.qo, 1, hkv, 152)
    assert slots == 0 and (np.diff(offsets) == 2).all()
    p = b.plan(lib)
    clean, lse = p.run(b.q, b.kv)
    assert p.check() == 0
    b.check(clean, lse, rows=8)
    page, slot = int(b.indices[-1]), (ctx + n - 1) % 16
    kv = b.kv.clone()
    kv[page, 1, slot, 0, 5] = float("inf")
    o, l = p.run(b.q, kv)
    assert p.check() == 0  # no wait gave up
    assert torch.equal(l, lse) and not torch.isfinite(o[-1, 0, 5])
    o[-1, 0, 5] = clean[-1, 0, 5]
    # all rows but those of the last block in head 0 are not touched at all
    assert torch.equal(o[:, 1:], clean[:, 1:]) and torch.equal(o[:-256, 0], clean[:-256, 0])
    # the token stands in a tile that the block's second 128 rows alone take part in;
    # computed again, they have other roundings
    again = (o[-256:, 0] != clean[-256:, 0]).any(-1)
    assert (ctx + n - 1) // 128 > (ctx + n - 129) // 128
    assert not again[:128].any() and again[128:255].sum() > 100
    b.check(o, l, rows=40)

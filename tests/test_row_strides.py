"""Strides of q that the tensor copies cannot take are refused by prefill and weights
before anything is launched: a mixed batch's first kernel too."""
import ctypes

import pytest
import torch

from tests.test_prefill import BF16, Batch
from tests.test_weights import fresh, plan


@pytest.mark.gpu
@pytest.mark.parametrize("token,head", [(2 ** 39, 128), (1024, 2 ** 39), (2 ** 62, 128), (0, 128), (1024, -128),
                                        (1020, 128)])
def test_strides_out_of_range(lib, cuda, token, head):
    b = Batch([40, 300], [1, 60], 8, 2, 128, BF16, seed=3)  # few columns, and many
    L = lib.library()
    rows = (ctypes.c_int64 * 3)(b.q.data_ptr(), token, head)
    o, lse = torch.full_like(b.q, 7), torch.zeros((b.T, 8), device=cuda)
    w = fresh(b)
    before, pf, wp = w.clone(), b.plan(lib), plan(b, lib)
    assert L.fa_prefill_run(pf._h, ctypes.addressof(rows), b.kv.data_ptr(), b.num_pages, 0.0, 1.0, 1.0,
                            o.data_ptr(), lse.data_ptr(), None) == -1
    assert L.fa_weights_run(wp._h, ctypes.addressof(rows), b.kv.data_ptr(), b.num_pages, 0.0, 1.0,
                            lse.data_ptr(), w.data_ptr(), None) == -1
    torch.cuda.synchronize()
    assert (o == 7).all() and not lse.any() and torch.equal(w, before)


@pytest.mark.gpu
def test_strides_that_are_never_taken(lib, cuda):
    b = Batch([300], [1], 1, 1, 128, BF16, seed=3)
    L = lib.library()
    o, lse = b.plan(lib).run(b.q, b.kv)
    rows = (ctypes.c_int64 * 3)(b.q.data_ptr(), 2 ** 62, -8)
    o2 = torch.empty_like(o)
    pf = b.plan(lib)
    assert L.fa_prefill_run(pf._h, ctypes.addressof(rows), b.kv.data_ptr(), b.num_pages, 0.0, 1.0, 1.0,
                            o2.data_ptr(), None, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, o2)

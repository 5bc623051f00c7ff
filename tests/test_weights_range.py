"""Accumulated weights: rows that count for nothing, whatever their q holds.  Bounds as
in test_weights.py."""
import numpy as np
import pytest

from tests.test_prefill import BF16, F16, Batch
from tests.test_weights import check, exact_lse, fresh, plan


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,d,hq,hkv,ctx,new", [
    (BF16, 128, 8, 8, 300, 5), (F16, 64, 8, 2, 300, 2), (BF16, 128, 8, 2, 300, 90),
    (F16, 64, 4, 4, 500, 300), (BF16, 64, 8, 1, 100, 3)])
def test_rows_of_minus_infinity_add_nothing(lib, cuda, dtype, d, hq, hkv, ctx, new, value):
    """A padded batch: rows whose lse is -inf hold anything in q."""
    b = Batch([ctx], [new], hq, hkv, d, dtype, seed=33)
    lse, w = exact_lse(b), fresh(b)
    dead = np.unique([0, new // 2, new - 1])
    lse[dead] = -float("inf")
    lse[new // 3, 0] = -float("inf")  # one head of a row alone
    before, p = w.clone(), plan(b, lib)
    q = b.q.clone()
    q[dead] = value
    q[new // 3, 0] = value
    p.run(q, b.kv, lse, w)
    check(b, w, before, lse)

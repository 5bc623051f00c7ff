"""Prompt attention whose weights lie far apart, in f16; bounds as in
test_prefill.py."""
import numpy as np
import pytest
import torch

from tests.test_prefill import F16, Batch


def flat_batch(n, d, drop, big, dtype=F16):
    """A prompt whose token 0 has logit 0 and value 0, all others a logit of -drop
    log2 units and values `big`."""
    b = Batch([0], [n], 1, 1, d, dtype, garbage=0.0)
    t = torch.arange(n, device="cuda")
    page = b.indices.long()[t // 16]
    b.q.zero_()
    b.q[..., 0] = 1
    b.kv.zero_()
    # logits sm_scale q k = k / 8, of the k that the cache holds
    k = round(-drop * np.log(2) * 8 * 32) / 32
    b.kv[page[1:], 0, t[1:] % 16, 0, 0] = k
    b.kv[page[1:], 1, t[1:] % 16, 0] = big
    return b


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,drop", [(256, 25.5), (256, 20.0), (200, 28.0), (256, 14.5), (500, 23.0)])
def test_small_f16_weights_count(lib, cuda, n, drop, d):
    """Weights of 2^-drop of the largest on large values.  A weight is held to half a
    step or, being subnormal, to 2^-25 / 2^7 of the largest: 2^-32 sum_t |v_t|."""
    big = 30000.0
    b = flat_batch(n, d, drop, big)
    o, lse = b.plan(lib).run(b.q, b.kv, sm_scale=0.125)
    rows = torch.arange(1, n + 1, device=cuda, dtype=torch.float64)  # tokens a row sees
    k = float(b.kv[b.indices.long()[0], 0, 1, 0, 0].double()) * 0.125
    w = np.exp(k)
    want = (rows - 1) * w * big / (1 + (rows - 1) * w)
    # the factor sm_scale log2 e and the product are floats: 2^-23 of k in the
    # exponent; 2^-21 for the exponential and the sums
    err = 2.0 ** -22 * abs(k) + 2.0 ** -20
    bound = want * (2 * 2.0 ** -11 + err) + 2.0 ** -32 * (rows - 1) * big + 2.0 ** -25
    got = o[:, 0].double()
    bad = ~((got - want[:, None]).abs() <= bound[:, None] * 1.001)
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], want[bad.nonzero()[:4, 0]])


@pytest.mark.gpu
def test_f16_logits_that_leap(lib, cuda):
    """Maxima that rise by 0 to 20 log2 units a tile: weights stay within f16."""
    for step in (0.5, 4.0, 7.9, 8.1, 16.0):
        b = Batch([700], [90], 2, 1, 64, F16, seed=6)
        t = torch.arange(790, device=cuda)
        page = b.indices.long()[t // 16]
        b.q.zero_()
        b.q[..., 0] = 1
        b.kv[page, 0, t % 16, 0] = 0
        b.kv[page, 0, t % 16, 0, 0] = ((t // 128) * step * np.log(2) * 8).to(F16)
        b.kv[page, 1, t % 16, 0] *= 1000
        o, lse = b.plan(lib).run(b.q, b.kv)
        b.check(o, lse)

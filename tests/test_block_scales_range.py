"""Block-scaled decode where scales and softmax weights are far apart: low weights
beside ignored pages of large V scales, and V scales over fp32's whole range.

Low weights.  Every A consecutive pages of a period of T pages are ignored by the
softmax (weight 0) and have a V scale `ratio` times the others'; the A pages after
them hold one attended token each (weight 1); the other n tokens an attended one
have the same weight e, about 2^-19, and V is of one sign.  The f16 weights of
P.V keep e to half a step of f16's subnormals, 2^-25, as they do under a
per-tensor scale, whatever the ratio.  Tolerance, relative to o: half a step of
the output's type; 2^-12 for the f16 rounding of normal weights; n * 2^-25 in
the numerator and as much in the per-tensor kernel's denominator, times
the largest |v| over the mean, below 2.  (What it catches: with the weights below
2^-25 of the ignored pages' scale gone, o is off by n e = 0.8 % and more.)
"""
import math

import numpy as np
import pytest
import torch

E4M3 = torch.float8_e4m3fn
BF16, F16 = torch.bfloat16, torch.float16
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}

pytestmark = pytest.mark.gpu


class Pattern:
    """Pages of the pattern above, shared by all requests."""

    def __init__(self, A, T, pages, hkv, d, ratio, e, device):
        self.hkv, self.d, self.A, self.T = hkv, d, A, T
        g = torch.Generator(device=device).manual_seed(1)
        raw = torch.empty((pages, 2, 16, hkv, d), dtype=torch.uint8, device=device)
        raw[:, 0] = 0xb8                                    # K code -1
        phase = torch.arange(pages, device=device) % T
        self.ignored, att = phase < A, (phase >= A) & (phase < 2 * A)
        raw[self.ignored, 0] = 0xfe                         # K code -448
        raw[att, 0, 0] = 0                                  # K code 0
        raw[:, 1] = torch.randint(0x38, 0x40, raw[:, 1].shape, generator=g, device=device,
                                  dtype=torch.uint8)        # V codes 1 .. 1.875
        self.kv = raw.view(E4M3)
        self.ks = torch.full((pages, hkv), 1.0 / d, device=device)
        self.vs = torch.full((pages, hkv), 2.0 ** -5, device=device)
        self.vs[self.ignored] *= ratio
        self.sm_scale = -math.log(e)                        # a low token's logit is -sm_scale
        w = torch.full((pages, 16), e, dtype=torch.float64, device=device)
        w[self.ignored] = 0
        w[att, 0] = 1
        self.w = w.flatten()

    def expect(self, repeats, drop=0):
        """(o [hkv, d], lse) over `repeats` passes over the pages, but for the
        last `drop` tokens."""
        v = self.kv[:, 1].double().flatten(0, 1) * 2.0 ** -5
        num, den = torch.einsum("t,thd->hd", self.w, v), self.w.sum()
        end = len(self.w) - drop
        tail = torch.einsum("t,thd->hd", self.w[end:], v[end:])
        num, den = num * repeats - tail, den * repeats - self.w[end:].sum()
        return num / den, math.log(float(den))

    def check(self, o, lse, dtype, repeats=1, drop=0, extra=0.0):
        """o [..., hkv * group, d]"""
        ro, rl = self.expect(repeats, drop)
        got = o.double().unflatten(-2, (self.hkv, -1))
        n = 16 * self.T / self.A
        tol = (HALF[dtype] + extra + 2.0 ** -12 + 2 * n * 2.0 ** -25) * ro
        err = (got - ro[:, None]).abs().amax(dim=tuple(range(got.dim() - 3)) + (-2,))
        assert (err <= tol).all(), float((err / ro).max())
        assert float((lse.double() - rl).abs().max()) <= 1e-4


E = [0.99 * 2.0 ** -19, 1.5 * 2.0 ** -18, 1.45 * 2.0 ** -20]


@pytest.mark.parametrize("e", E)
@pytest.mark.parametrize("ratio", [1.0, 32.0, 64.0, 2.0 ** -5])
@pytest.mark.parametrize("d,group,A,batch", [(128, 1, 4, 320), (128, 8, 4, 320), (64, 8, 16, 96),
                                             (64, 4, 24, 240)])
def test_low_weights_page_split(lib, cuda, d, group, A, batch, ratio, e):
    T = 1024 * A
    s = Pattern(A, T, T + T // 2, 2, d, ratio, e, cuda)
    pages = s.kv.shape[0]
    indices = torch.arange(pages, dtype=torch.int32, device=cuda).repeat(batch)
    p = lib.plan(np.arange(batch + 1) * pages, indices, [16] * batch, 2 * group, 2, d, 16,
                 q_data_type=F16, kv_data_type=E4M3)
    q = torch.ones((batch, 2 * group, d), dtype=F16, device=cuda)
    o, lse = p.run_block_scales(q, s.kv, s.ks, s.vs, sm_scale=s.sm_scale)
    s.check(o, lse, F16)
    if ratio == 1 and d == 128 and group > 1:   # the per-tensor kernel, on the tensor cores
        o, _ = p.run(q, s.kv, k_scale=1.0 / d, v_scale=2.0 ** -5, sm_scale=s.sm_scale)
        s.check(o, lse, F16)
    assert p.check() == 0


@pytest.mark.parametrize("e", E)
@pytest.mark.parametrize("ratio", [1.0, 32.0, 64.0])
@pytest.mark.parametrize("count", [2, 3, 4])
def test_low_weights_column_split(lib, cuda, count, ratio, e):
    batch, group, d, T = 256, 8, 128, 1024
    s = Pattern(1, T, 2 * T, 2, d, ratio, e, cuda)
    pages = s.kv.shape[0]
    indices = torch.arange(pages, dtype=torch.int32, device=cuda).repeat(batch)
    p = lib.plan_ragged_q(np.arange(batch + 1) * pages, indices, [16] * batch,
                          np.arange(batch + 1) * count, 2 * group, 2, d, 16, q_data_type=BF16,
                          kv_data_type=E4M3)
    q = torch.ones((batch * count, 2 * group, d), dtype=BF16, device=cuda)
    o, lse = p.run_block_scales(q, s.kv, s.ks, s.vs, sm_scale=s.sm_scale)
    for i in range(count):
        s.check(o[i::count], lse[i::count], BF16, drop=count - 1 - i)
    assert p.check() == 0


@pytest.mark.parametrize("e", E)
@pytest.mark.parametrize("ratio", [1.0, 32.0, 64.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_low_weights_cascade(lib, cuda, dtype, ratio, e):
    batch, group, d, T, repeats = 64, 8, 128, 1024, 20
    s = Pattern(1, T, 2 * T, 2, d, ratio, e, cuda)
    pages = s.kv.shape[0]
    prefix = torch.arange(pages, dtype=torch.int32, device=cuda).repeat(repeats)
    p = lib.cascade_plan(prefix, [0] * (batch + 1), prefix[:0], [16] * batch, 2 * group, 2, d, 16,
                         q_data_type=dtype, kv_data_type=E4M3)
    q = torch.ones((batch, 2 * group, d), dtype=dtype, device=cuda)
    o, lse = p.run_block_scales(q, s.kv, s.ks, s.vs, sm_scale=s.sm_scale)
    s.check(o, lse, dtype, repeats=repeats)
    assert p.check() == 0

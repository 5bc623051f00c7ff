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


# ---------------------------------------------------------------- V scales far apart

def tiny_and_ordinary(order, n, tiny=2.0 ** -120):
    """Per page, the factor of V's values: 1, or `tiny` (2^-120: values near 1e-36,
    whose block scale is 2^-126)."""
    f = np.ones(n)
    third = n // 3
    if order == "before":
        f[:third] = tiny
    elif order == "between":
        f[third:2 * third] = tiny
    elif order == "after":
        f[2 * third:] = tiny
    elif order == "one":
        f[n // 2] = tiny
    else:                                     # each smaller than the one before
        f = 2.0 ** (-np.linspace(0, 120, n))
    return f


def appended(lib, lengths, order, hq, hkv, d, device, seed, tiny=2.0 ** -120):
    """A cache written by run_block_scales, V's pages of such values."""
    from tests.test_append import Batch
    b = Batch([0] * len(lengths), lengths, hq, hkv, d, BF16, E4M3, seed=seed, device=device)
    v = torch.cat([torch.randn((n, hkv, d), device=device)
                   * torch.from_numpy(np.repeat(tiny_and_ordinary(order, (n + 15) // 16, tiny), 16)[:n])
                   .float().to(device)[:, None, None] for n in lengths]).to(BF16)
    k = torch.randn((b.T, hkv, d), device=device).to(BF16)
    ks, vs = (torch.full((b.num_pages, hkv), float("nan"), device=device) for _ in range(2))
    b.plan(lib).run_block_scales(k, v, b.kv, ks, vs)
    assert float(vs.nan_to_num(1.0).min()) <= tiny * 2.0 ** -5
    return b, ks, vs


def reference(b, ks, vs, q, rows, prefix=0, repeats=1):
    """(o, lse, sum w |v|) in 64 bits over the dequantised cache, its first `prefix`
    tokens taken `repeats` times."""
    o, lse, mag = [], [], []
    at = 0
    for i, r in enumerate(rows):
        n = int(b.new[i])
        ids = torch.from_numpy(b.ids[b.indptr[i]:b.indptr[i + 1]].astype(np.int64)).to(q.device)
        kv = b.kv[ids].double()
        k = (kv[:, 0] * ks[ids].double()[:, None, :, None]).flatten(0, 1)[:n]
        v = (kv[:, 1] * vs[ids].double()[:, None, :, None]).flatten(0, 1)[:n]
        x = q[at:at + r].double().unflatten(1, (b.hkv, -1))          # [r, hkv, g, d]
        w = torch.einsum("rhgd,nhd->rhgn", x, k) * b.d ** -0.5
        w[..., :prefix] += math.log(repeats)
        seen = torch.arange(n, device=q.device) <= n - r + torch.arange(r, device=q.device)[:, None]
        w = w.masked_fill(~seen[:, None, None], -math.inf)
        lse.append(torch.logsumexp(w, -1).flatten(1))
        w = torch.softmax(w, -1)
        o.append(torch.einsum("rhgn,nhd->rhgd", w, v).flatten(1, 2))
        mag.append(torch.einsum("rhgn,nhd->rhgd", w, v.abs()).flatten(1, 2))
        at += r
    return torch.cat(o), torch.cat(lse), torch.cat(mag)


def close(o, lse, ref, extra=0.0):
    """As the block-scale tests: half a step of the output, 3 * 2^-11 for the f16
    weights and 2e-4 for the logits, of sum w |v|."""
    ro, rl, mag = ref
    assert torch.isfinite(o).all()
    err = (o.double().reshape(ro.shape) - ro).abs()
    tol = HALF[o.dtype] * ro.abs() + (3 * 2.0 ** -11 + 2e-4 + extra) * mag
    assert (err <= tol * 1.01 + 1e-38).all(), float((err / tol).max())
    assert float((lse.double().reshape(rl.shape) - rl).abs().max()) <= 1e-4


ORDERS = ["before", "between", "after", "one", "falling"]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("d,group", [(128, 1), (128, 8), (64, 4), (64, 8)])
def test_appended_tiny_values_page_split(lib, cuda, d, group, order):
    lengths = [700, 3000, 16, 1500]
    b, ks, vs = appended(lib, lengths, order, 2 * group, 2, d, cuda, 1)
    p = lib.plan(b.indptr, b.indices, b.last, 2 * group, 2, d, 16, q_data_type=BF16,
                 kv_data_type=E4M3)
    q = torch.randn((4, 2 * group, d), device=cuda).to(BF16)
    o, lse = p.run_block_scales(q, b.kv, ks, vs)
    close(o, lse, reference(b, ks, vs, q, [1] * 4))
    assert p.check() == 0


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("counts", [[4, 4, 4, 4], [2, 1, 2, 1], [3, 1, 0, 2]])
def test_appended_tiny_values_column_split(lib, cuda, counts, order):
    lengths = [700, 3000, 16, 1500]
    b, ks, vs = appended(lib, lengths, order, 16, 2, 128, cuda, 2)
    p = lib.plan_ragged_q(b.indptr, b.indices, b.last, np.concatenate([[0], np.cumsum(counts)]),
                          16, 2, 128, 16, q_data_type=BF16, kv_data_type=E4M3)
    q = torch.randn((sum(counts), 16, 128), device=cuda).to(BF16)
    o, lse = p.run_block_scales(q, b.kv, ks, vs)
    close(o, lse, reference(b, ks, vs, q, counts))
    assert p.check() == 0


@pytest.mark.parametrize("order", ORDERS)
def test_appended_tiny_values_cascade(lib, cuda, order):
    """The prefix is one request of the append, its pages many times over (a CTA
    then holds several changes of scale); the cascade's requests have it, and
    one page more, the last of another."""
    b, ks, vs = appended(lib, [2400, 16], order, 16, 2, 128, cuda, 3)
    batch, repeats = 20, 64
    own = b.indices[150:151].repeat(batch)
    p = lib.cascade_plan(b.indices[:150].repeat(repeats), np.arange(batch + 1), own, [16] * batch,
                         16, 2, 128, 16, q_data_type=BF16, kv_data_type=E4M3)
    q = torch.randn((batch, 16, 128), device=cuda).to(BF16)
    o, lse = p.run_block_scales(q, b.kv, ks, vs)
    b.indptr, b.new = np.array([0, 151]), np.array([2416])  # all 151 pages as one request
    refs = [reference(b, ks, vs, q[i:i + 1], [1], 2400, repeats) for i in range(batch)]
    close(o, lse, [torch.cat(x) for x in zip(*refs)], extra=HALF[BF16])
    assert p.check() == 0


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("counts", [None, [4, 3]])
def test_attended_tiny_values_beside_ignored_ordinary_ones(lib, cuda, counts, first):
    """The other way round: the softmax ignores the ordinary pages (weight 0), and
    what is left are values 2^64 below theirs, in full precision."""
    lengths, hq, hkv, d = [640, 1600], 16, 2, 128
    b, ks, vs = appended(lib, lengths, "after" if first else "before", hq, hkv, d, cuda, 4,
                         tiny=2.0 ** -64)
    q = torch.rand((sum(counts) if counts else 2, hq, d), device=cuda).add_(0.5).to(BF16)
    ids = torch.from_numpy(b.ids[:b.indptr[2]].astype(np.int64)).to(cuda)
    raw = b.kv.view(torch.uint8)
    raw[ids, 0] = raw[ids, 0] & 0x3f                # K codes 0 .. 1.9
    ks[ids] = 2.0 ** -6
    ordinary = ids[(vs[ids] > 2.0 ** -40).all(-1)]
    raw[ordinary, 0] = 0xfe                         # and -448
    ks[ordinary] = 4.0
    args = (hq, hkv, d, 16)
    if counts:
        p = lib.plan_ragged_q(b.indptr, b.indices, b.last, [0, 4, 7], *args, q_data_type=BF16,
                              kv_data_type=E4M3)
    else:
        p = lib.plan(b.indptr, b.indices, b.last, *args, q_data_type=BF16, kv_data_type=E4M3)
    o, lse = p.run_block_scales(q, b.kv, ks, vs)
    ref = reference(b, ks, vs, q, counts or [1, 1])
    assert 0 < float(ref[0].abs().max()) < 1e-16
    err = (o.double().reshape(ref[0].shape) - ref[0]).abs()
    tol = HALF[BF16] * ref[0].abs() + (3 * 2.0 ** -11 + 2e-4) * ref[2]
    assert (err <= tol * 1.01).all(), float((err / tol).max())

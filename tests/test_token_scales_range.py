"""Decode over per-token scales as run_token_scales writes them, where V's values
are small, large or far apart: the f16 weights of P.V keep what they have under
scales near 1, since o is kept in units of a page's scale.  Against 64 bits over
the dequantised cache; per element half a step of the output, 3 * 2^-11 for
weights, weights times scales and their sum, and 2e-4 for the logits, of
sum w |v|; where scales lie far apart also 2^-25 of a page's largest |v| for each of
its tokens' weight, half a step of f16's subnormals.
"""
import math

import numpy as np
import pytest
import torch

from tests.test_append import BF16, E4M3, F16, Batch

HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}

pytestmark = pytest.mark.gpu


def written(lib, lengths, factor, hq, hkv, dtype, device, seed):
    """A cache of `lengths` written by run_token_scales, NaN where nothing was; V's
    tokens times factor(n)."""
    b = Batch([0] * len(lengths), lengths, hq, hkv, 128, dtype, E4M3, seed=seed, device=device)
    b.kv.view(torch.uint8).fill_(0x7f)
    f = np.concatenate([factor(n) for n in lengths])
    v = torch.randn((b.T, hkv, 128), device=device).double()
    v = (v * torch.from_numpy(f).to(device)[:, None, None]).to(dtype)
    k = torch.randn((b.T, hkv, 128), device=device).to(dtype)
    ks, vs = (torch.full((b.num_pages, hkv, 16), float("nan"), device=device) for _ in range(2))
    b.plan(lib).run_token_scales(k, v, b.kv, ks, vs)
    return b, ks, vs


def check(lib, b, ks, vs, dtype, seed=0):
    p = lib.plan(b.indptr, b.indices, b.last, b.hq, b.hkv, 128, 16, q_data_type=dtype,
                 kv_data_type=E4M3)
    assert p.info["tensor_cores"] == 1
    g = torch.Generator(device=b.kv.device).manual_seed(seed)
    q = torch.randn((len(b.new), b.hq, 128), generator=g, device=b.kv.device).to(dtype)
    o, lse = p.run_token_scales(q, b.kv, ks, vs)
    torch.cuda.synchronize()
    assert p.check() == 0 and torch.isfinite(o).all()
    for i, n in enumerate(b.new):
        ids = torch.from_numpy(b.ids[b.indptr[i]:b.indptr[i + 1]].astype(np.int64)).to(q.device)
        s = torch.stack([ks, vs], 1)[ids].double().transpose(2, 3)[..., None]
        kv = (b.kv[ids].double() * s).transpose(1, 2).flatten(0, 1)[:n]       # [n, 2, hkv, d]
        x = q[i].double().unflatten(0, (b.hkv, -1))
        w = torch.einsum("hgd,nhd->hgn", x, kv[:, 0]) / math.sqrt(128)
        rl = torch.logsumexp(w, -1).flatten()
        w = torch.softmax(w, -1)
        ro = torch.einsum("hgn,nhd->hgd", w, kv[:, 1]).flatten(0, 1)
        mag = torch.einsum("hgn,nhd->hgd", w, kv[:, 1].abs()).flatten(0, 1)
        # weights that are subnormal in f16: each at most 2^-25 of its page's largest |v|
        top = kv[:, 1].abs().amax(-1)
        pages = torch.nn.functional.pad(top, (0, 0, 0, -int(n) % 16)).view(-1, 16, b.hkv).amax(1)
        tail = (pages.sum(0) * 16 * 2.0 ** -25 * float(w.amax(-1).max())).repeat_interleave(
            b.hq // b.hkv)[:, None]
        tol = HALF[dtype] * ro.abs() + (3 * 2.0 ** -11 + 2e-4) * mag + tail
        if dtype == F16:
            tol = tol + 2.0 ** -25
        err = (o[i].double() - ro).abs()
        assert (err <= 1.01 * tol + 1e-38).all(), (i, float((err / tol).max()))
        assert float((lse[i].double() - rl).abs().max()) <= 2.0 ** -11 + 1e-4


LENGTHS = [700, 1, 16, 3000, 45]


@pytest.mark.parametrize("log2", [-100, -60, -24, -17, -10, 0, 10, 40])
@pytest.mark.parametrize("group", [2, 4, 8])
def test_values_of_any_size(lib, cuda, group, log2):
    b, ks, vs = written(lib, LENGTHS, lambda n: np.full(n, 2.0 ** log2), 2 * group, 2, BF16, cuda,
                        group)
    check(lib, b, ks, vs, BF16)


@pytest.mark.parametrize("log2", [-10, 0, 10])
def test_values_of_any_size_f16(lib, cuda, log2):
    b, ks, vs = written(lib, LENGTHS, lambda n: np.full(n, 2.0 ** log2), 8, 2, F16, cuda, 3)
    check(lib, b, ks, vs, F16)


def steps(order):
    def factor(n):
        f = np.ones(n)
        third = n // 3
        if order == "before":
            f[:third] = 2.0 ** -90
        elif order == "between":
            f[third:2 * third] = 2.0 ** -90
        elif order == "after":
            f[2 * third:] = 2.0 ** -90
        elif order == "falling":
            f = 2.0 ** (-np.linspace(0, 90, n))
        elif order == "rising":
            f = 2.0 ** (-np.linspace(90, 0, n))
        else:
            f = 2.0 ** np.rint(np.random.default_rng(1).uniform(-12, 12, n))
        return f
    return factor


@pytest.mark.parametrize("order", ["before", "between", "after", "falling", "rising", "mixed"])
@pytest.mark.parametrize("group", [2, 8])
def test_values_far_apart(lib, cuda, group, order):
    b, ks, vs = written(lib, LENGTHS, steps(order), 2 * group, 2, BF16, cuda, 5 + group)
    check(lib, b, ks, vs, BF16)


def test_zeros_among_them(lib, cuda):
    """Pages and tokens of zeros, whose scale is 0."""
    def factor(n):
        f = np.ones(n) * 2.0 ** -20
        f[::3] = 0
        f[32:64] = 0
        return f
    b, ks, vs = written(lib, LENGTHS, factor, 8, 2, BF16, cuda, 11)
    check(lib, b, ks, vs, BF16)

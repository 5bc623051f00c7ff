"""Accumulated weights beyond a CTA's first job: batches of many runs, in both kernels.
Bounds as in test_weights.py."""
import numpy as np
import pytest
import torch

from tests.test_prefill import BF16, E4M3, F16, Batch
from tests.test_weights import check, exact_lse, fresh, plan


def scales_of(b, mode, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda") * 0.1 + 0.001  # noqa: E731
    if mode == "token":
        s = rand(b.num_pages, b.hkv, 16)
        return s, lambda page, slot: s.double()[page, :, slot]
    if mode == "block":
        s = rand(b.num_pages, b.hkv)
        return s, lambda page, slot: s.double()[page]
    if mode == "head":
        s = rand(b.hkv)
        return s, lambda page, slot: s.double().expand(len(page), b.hkv)
    return None, None


def run_and_check(lib, b, mode):
    s, of = scales_of(b, mode)
    lse, w = exact_lse(b, of), fresh(b)
    before, p = w.clone(), plan(b, lib)
    args = (b.q, b.kv, lse, w)
    if s is None:
        p.run(*args)
    else:
        getattr(p, f"run_{mode}_scales")(*args, s)
    assert p.check() == 0
    check(b, w, before, lse, of)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv,mode,d,hq,hkv", [
    (BF16, None, None, 128, 32, 8), (F16, None, None, 64, 16, 8), (BF16, E4M3, "token", 128, 16, 8),
    (BF16, E4M3, "block", 64, 32, 8), (F16, E4M3, "head", 128, 32, 8), (F16, E4M3, "token", 64, 16, 8)])
def test_many_jobs_a_cta(lib, cuda, dtype, kv, mode, d, hq, hkv):
    """24 requests of 1000-5000 tokens: three jobs and more a CTA, of one block of
    tokens and of two in turn, of one tile of columns and of several."""
    r = np.random.default_rng(d + hq)
    new = r.integers(3, 41, 24)
    new[5] = 150
    b = Batch(r.integers(1000, 5001, 24) - new, new, hq, hkv, d, dtype, kv, seed=hq)
    assert (-(-((b.total + 15) // 16) // 16)).sum() * hkv > 3 * 152
    run_and_check(lib, b, mode)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv,mode,d,hq,hkv", [
    (BF16, None, None, 128, 32, 8), (F16, None, None, 64, 64, 8), (BF16, E4M3, "block", 128, 8, 8),
    (F16, E4M3, "token", 64, 16, 8)])
def test_decode_steps_of_long_runs(lib, cuda, dtype, kv, mode, d, hq, hkv):
    """One row a request: runs of 64 pages, eight a warp, and their odd ends."""
    r = np.random.default_rng(d)
    b = Batch(r.integers(1000, 4001, 44), [1] * 44, hq, hkv, d, dtype, kv, seed=hq)
    assert int(b.indptr[-1]) * hkv >= 64 * 4 * 152
    run_and_check(lib, b, mode)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,mode", [(None, None), (E4M3, "token")])
def test_mixed_steps_of_both_kernels(lib, cuda, kv, mode):
    """Single rows, windows and chunks in one batch: each kernel passes its CTAs more
    than once."""
    r = np.random.default_rng(5)
    new = np.where(np.arange(64) % 2, 1, r.integers(3, 70, 64))
    b = Batch(r.integers(500, 6000, 64) - new % 100, new, 32, 8, 128, BF16, kv, seed=6)
    run_and_check(lib, b, mode)

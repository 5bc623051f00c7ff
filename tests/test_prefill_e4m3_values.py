"""Prompt attention over E4M3 caches: values that are not finite at tokens that a row
does not see, under every kind of scale.  Bounds as in test_prefill.py."""
import pytest
import torch

from tests.test_prefill import BF16, E4M3, Batch


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,new", [([40], [90]), ([0], [300]), ([20000], [40])])
@pytest.mark.parametrize("mode", ["tensor", "head", "token", "token_scale", "block"])
def test_e4m3_values_that_a_row_does_not_see(lib, cuda, mode, ctx, new):
    """A NaN code in V, or a scale of NaN, at a token in the middle of the prompt:
    rows before it have their finite results."""
    hq, hkv, d, n = 8, 2, 128, new[0]
    b = Batch(ctx, new, hq, hkv, d, BF16, E4M3, seed=15)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda") * 0.1 + 0.001  # noqa: E731
    at = n // 2
    page, slot = int(b.indices[(ctx[0] + at) // 16]), (ctx[0] + at) % 16
    inexact = False
    if mode == "tensor":
        s, run = [torch.full((2,), 0.125, device=cuda), torch.full((2,), 0.25, device=cuda)], None
        of = lambda half, p, t: s[half].double().expand(len(p), 2)  # noqa: E731
    elif mode == "head":
        s, run = [rand(2), rand(2)], "run_head_scales"
        of = lambda half, p, t: s[half].double().expand(len(p), 2)  # noqa: E731
    elif mode == "block":
        s, run = [torch.exp2(torch.floor(rand(b.num_pages, 2) * 90) - 9) for _ in range(2)], "run_block_scales"
        of = lambda half, p, t: s[half].double()[p]  # noqa: E731
    else:
        s, run, inexact = [rand(b.num_pages, 2, 16) for _ in range(2)], "run_token_scales", True
        of = lambda half, p, t: s[half].double()[p, :, t]  # noqa: E731
    p = b.plan(lib)

    def attend(kv, s):
        if run is None:
            return p.run(b.q, kv, k_scale=0.125, v_scale=0.25)
        return getattr(p, run)(b.q, kv, *s)

    clean, lse = attend(b.kv, s)
    b.check(clean, lse, of, inexact, rows=30)
    kv, bad_s = b.kv.clone(), [x.clone() for x in s]
    if mode == "token_scale":
        bad_s[1][page, 0, slot] = float("nan")
        dims = slice(None)
    else:
        kv.view(torch.uint8)[page, 1, slot, 0, 5] = 127
        dims = 5
    o, l = attend(kv, bad_s)
    assert p.check() == 0 and torch.equal(l, lse)
    G = hq // hkv
    assert torch.isnan(o[at:, :G, dims]).all()
    o[at:, :G, dims] = clean[at:, :G, dims]
    b.check(o, l, of, inexact, rows=30)
    assert torch.equal(o[at:], clean[at:]) and torch.equal(o[:, G:], clean[:, G:])

"""Prompt attention over E4M3 caches: V's scales cost no rounding of their own, but for
those per block that are no powers of two (append writes powers of two).

The measure.  Rounding to bf16 (steps of 2^-7 in [1, 2)) is off by 2^-7 / sqrt(12) of the
step's base, rms; over mantissas spread evenly in their logarithm (mean of 1 / x^2 =
(1 - 1/4) / (2 ln 2) = 0.541) that is R = 2^-7 sqrt(0.541 / 12) = 1.66e-3 of the value.
Weights are rounded once, independently, and o once: the expected square of o's error
is R^2 (sum_t (w_t v_t)^2 + o^2).  Rounding V's elements as well would make it
R^2 (2 sum_t (w_t v_t)^2 + o^2), half as much again where values have either sign.  The mean
over 10^5 elements and more of o lies within 15 % of the expectation (the elements of
a row share their weights' roundings, so some 10^3 are independent: 4 % for one
deviation; mantissas are not quite spread so, and logits are 2^-18 off)."""
import numpy as np
import pytest
import torch

from tests.test_prefill import BF16, E4M3, Batch

R2 = (2.0 ** -7) ** 2 * 0.541 / 12


def mean_squares(b, o, scale_of, roundings=1):
    """The mean square of o's error, and what the roundings make of it: `roundings` of each
    weight times value, and one of o."""
    got, want = [], []
    G, sm = b.hq // b.hkv, b.d ** -0.5
    kv = b.kv.double()
    for i in range(len(b.total)):
        n, L = int(b.new[i]), int(b.total[i])
        t = torch.arange(L, device="cuda")
        page = b.indices[b.indptr[i]:b.indptr[i + 1]].long()[t // 16]
        k = kv[page, 0, t % 16] * scale_of(0, page, t % 16)[..., None]
        v = kv[page, 1, t % 16] * scale_of(1, page, t % 16)[..., None]
        a = int(b.qo[i])
        seen = t[None, :] <= (L - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(b.hq):
            s = (b.q[a:a + n, h].double() @ k[:, h // G].T * sm).masked_fill(~seen, -float("inf"))
            w = s.softmax(-1)
            x = w @ v[:, h // G]
            got.append(((o[a:a + n, h].double() - x) ** 2).mean())
            want.append((roundings * ((w ** 2) @ (v[:, h // G] ** 2)) + x ** 2).mean() * R2)
    return float(torch.stack(got).mean()), float(torch.stack(want).mean())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", ["head", "token", "block_any", "block"])
def test_one_rounding_of_weights_and_one_of_o(lib, cuda, mode, d):
    b = Batch([20, 300, 40], [60, 100, 200], 16, 4, d, BF16, E4M3, seed=17)
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda") * 0.1 + 0.02  # noqa: E731
    if mode == "head":
        s, run = [rand(4), rand(4)], "run_head_scales"
        of = lambda half, p, t: s[half].double().expand(len(p), 4)  # noqa: E731
    elif mode == "token":
        s, run = [rand(b.num_pages, 4, 16) for _ in range(2)], "run_token_scales"
        of = lambda half, p, t: s[half].double()[p, :, t]  # noqa: E731
    else:
        s, run = [rand(b.num_pages, 4) for _ in range(2)], "run_block_scales"
        if mode == "block":
            s = [torch.exp2(x.log2().floor()) for x in s]
        of = lambda half, p, t: s[half].double()[p]  # noqa: E731
    o, _ = getattr(b.plan(lib), run)(b.q, b.kv, *s)
    got, want = mean_squares(b, o, of, 2 if mode == "block_any" else 1)
    assert got <= 1.15 * want, (got / want, got, want)
    assert got >= 0.5 * want, (got / want, got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["token", "block"])
def test_scales_of_any_size(lib, cuda, mode):
    """V's scales from 2^-120 to 2^100, one size a kv head, with mantissas next to 1 and
    next to 2, and 0: the bounds of test_prefill.py on each head."""
    size = torch.tensor([2.0 ** -120, 2.0 ** -60, 2.0 ** 40, 2.0 ** 100], device=cuda)
    b = Batch([20, 300], [60, 100], 8, 4, 128, BF16, E4M3, seed=18)
    g = torch.Generator(device="cuda").manual_seed(6)
    shape = (b.num_pages, 4, 16) if mode == "token" else (b.num_pages, 4)
    pick = torch.randint(0, 6, shape, generator=g, device="cuda")
    rest = torch.tensor([1.0, 1.0 + 2.0 ** -23, 2.0 - 2.0 ** -23, 1.5, 1.99, 0.0], device=cuda)[pick]
    ks = torch.full(shape, 0.05, device=cuda)
    vs = rest * (size[None, :, None] if mode == "token" else size[None])
    o, lse = getattr(b.plan(lib), f"run_{mode}_scales")(b.q, b.kv, ks, vs)
    assert torch.isfinite(o).all()
    b.check(o, lse, lambda half, p, t: ((ks, vs)[half].double()[p, :, t] if mode == "token"
                                        else (ks, vs)[half].double()[p]), inexact=True)

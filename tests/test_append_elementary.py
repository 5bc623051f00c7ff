"""Appended values against the same arithmetic in elementary operations: cos and
sin of a float64 angle rounded to fp32, products and sums rounded one by one in
fp32, one rounding into the stored type, codes by rn(x * (1 / scale)).  The append
kernel computes these very values, so q, K, codes and scales are equal bit for
bit but for a counted few.

How many may differ.  The kernel's cosines and sines are misrounded for one angle
in 10^5 (counted over 4 * 10^6 angles in quadruple precision).  The float64 angle
t f carries half a step, t f 2^-53 radians at most; a cosine or sine in [1/2, 1),
2^-24 apart from the next, is then misrounded with a probability of t f 2^-28, and
a smaller one moves an element by as much less as it is likelier to be: the
frequencies of 10000 ** (-j / (D / 2)) average 0.11, so that t = 2^17 gives 2^-14
an angle.  Each element takes two angles' values, and differs in fp32 for less than
2^-12 of them: 2^-10 is allowed.  In a type of fewer bits the fp32 values' last bit
decides with a probability of 2^-16 (bf16), 2^-13 (f16) and 2^-20 (E4M3): fewer
than one element in 10^7; two are allowed in a test's 10^6.
"""
import numpy as np
import pytest
import torch

from tests.test_append import BF16, E4M3, F16, F32, Batch, positions_of

pytestmark = pytest.mark.gpu


def rotated(x, positions, rotary):
    """x [T, H, D] in fp32, rotated with elementary operations."""
    y = x.float()
    if rotary is None:
        return y
    angle = torch.from_numpy(positions).to(x.device).double()[:, None, None] * torch.from_numpy(
        rotary.inv_freq).to(x.device)
    cos, sin = angle.cos().float(), angle.sin().float()
    n = rotary.rotary_dim // 2
    i = torch.arange(n, device=x.device)
    i1, i2 = (2 * i, 2 * i + 1) if rotary.interleaved else (i, i + n)
    a, b = y[..., i1], y[..., i2]
    out = y.clone()
    ac, bs, bc, as_ = a * cos, b * sin, b * cos, a * sin
    out[..., i1], out[..., i2] = ac - bs, bc + as_
    return out


def where(b, device):
    page, slot = (torch.tensor([p[i] for p in b.places()], device=device) for i in (2, 3))
    return page, slot


def differing(x, y):
    """Elements of x and y (no NaN) that are not equal."""
    return int((x.float() != y.float()).sum())


def codes(x, inv):
    return (x * inv).clamp(-448, 448).to(E4M3)


LENGTHS = ([0, 5, 15, 31, 0, 700, 1000], [1, 1, 17, 40, 300, 1, 33])


@pytest.mark.parametrize("offset", [0, 62000, 131072 - 1033])
@pytest.mark.parametrize("rotary_dim,interleaved", [(128, False), (128, True), (48, False)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_native(lib, cuda, dtype, rotary_dim, interleaved, offset):
    b = Batch(*LENGTHS, 16, 8, 128, dtype, dtype, seed=3)
    rot = lib.RotaryTable(rotary_dim, interleaved=interleaved)
    off = [offset] * len(b.ctx)
    q = b.plan(lib, rot, offset=off).run(b.k, b.v, b.kv, q=b.q)
    pos = positions_of(b, off)
    page, slot = where(b, cuda)
    n = 0
    for got, x in ((q, b.q), (b.kv[page, 0, slot], b.k)):
        n += differing(got, rotated(x, pos, rot).to(dtype))
    assert n <= (2.0 ** -10 * (b.q.numel() + b.k.numel()) if dtype == F32 else 2), n
    assert torch.equal(b.kv[page, 1, slot], b.v)


@pytest.mark.parametrize("mode", ["head", "token", "block"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_e4m3(lib, cuda, dtype, mode):
    b = Batch([0] * 7, LENGTHS[1], 16, 8, 128, dtype, E4M3, seed=4)
    rot = lib.RotaryTable(128)
    off = [62000] * 7
    p = b.plan(lib, rot, offset=off)
    pos = positions_of(b, off)
    page, slot = where(b, cuda)
    shape = {"head": (8,), "token": (b.num_pages, 8, 16), "block": (b.num_pages, 8)}[mode]
    ks, vs = (torch.full(shape, 0.03125, device=cuda) for _ in range(2))
    q = getattr(p, f"run_{mode}_scales")(b.k, b.v, b.kv, ks, vs, q=b.q)
    n = differing(q, rotated(b.q, pos, rot).to(dtype))
    for half, x, s in ((0, rotated(b.k, pos, rot), ks), (1, b.v.float(), vs)):
        amax = x.abs().amax(-1)
        if mode == "head":
            inv = 1 / s[:, None]
        elif mode == "token":
            got = s[page, :, slot]
            # by a tensor: torch turns a scalar divisor into a product with its reciprocal
            n_scale = differing(got, amax / torch.full_like(amax, 448))
            assert n_scale <= 2.0 ** -10 * got.numel(), n_scale
            inv = 1 / got[..., None]
        else:
            top = torch.zeros((b.num_pages, 8), device=cuda)
            top.index_reduce_(0, page, amax, "amax")
            e = torch.frexp(top / torch.full_like(top, 448))
            want = torch.ldexp(torch.ones_like(top), e.exponent - (e.mantissa == 0.5).int())
            used = torch.unique(page)
            assert torch.equal(s[used], want[used])
            inv = 1 / s[page][..., None]
        n += differing(b.kv[page, half, slot], codes(x, inv))
    assert n <= 2, n


def test_a_step_gives_the_attention_the_same_inputs(lib, cuda):
    """64 requests, a token each, as a decode step runs them: 262144 elements of
    q, of which a rotation off in fp32's last bit turns several."""
    rng = np.random.default_rng(1)
    ctx = rng.integers(512, 4096, 64)
    for seed in range(4):
        b = Batch(ctx, [1] * 64, 32, 8, 128, BF16, BF16, seed=seed)
        rot = lib.RotaryTable(128)
        q = b.plan(lib, rot).run(b.k, b.v, b.kv, q=b.q)
        pos = positions_of(b)
        page, slot = where(b, cuda)
        assert differing(q, rotated(b.q, pos, rot).to(BF16)) <= 1
        assert differing(b.kv[page, 0, slot], rotated(b.k, pos, rot).to(BF16)) <= 1


def test_a_table_changed_after_its_making(lib, cuda):
    """A RotaryTable whose frequencies were put in another type is read as doubles
    all the same, and one of another length is refused."""
    b = Batch([3, 0], [5, 20], 8, 2, 128, F32, F32, seed=6)
    rot = lib.RotaryTable(128)
    rot.inv_freq = rot.inv_freq.astype(np.float32)
    q = b.plan(lib, rot).run(b.k, b.v, b.kv, q=b.q)
    same = lib.RotaryTable(128, inv_freq=rot.inv_freq.astype(np.float64))
    assert torch.equal(q, b.plan(lib, same).run(b.k, b.v, b.kv, q=b.q))
    rot.inv_freq = rot.inv_freq[:32]
    with pytest.raises(ValueError):
        b.plan(lib, rot)

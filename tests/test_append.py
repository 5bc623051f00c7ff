"""Appending to the paged cache (plan_append) against the definition in 64
bits, and the refusals of its entry points.

Tolerances.  A stored value is rounded once from fp32: by half a step of its
type (bf16 2^-8, f16 2^-11 relative; an E4M3 code 2^-4 relative, 2^-10 in code
units below 2^-6), after an fp32 rotation.  The rotation's own error per
element: the angle carries the rounding of a fraction of a turn to fp32 (2^-25
half-turns, 9.4e-8 radians) and sincospi 1.5e-7, and two products and a sum
2^-23 of |x1| + |x2| - 4e-7 (|x1| + |x2|) bounds them together.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tests.helpers import as_bits

E4M3 = torch.float8_e4m3fn
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
ROT = 4e-7


# ---------------------------------------------------------------- the definition

class Batch:
    """A batch after its append: request i holds ctx[i] + new[i] tokens."""

    def __init__(self, ctx, new, hq, hkv, d, q_dtype, kv_dtype, seed=0, device="cuda", extra=3):
        rng = np.random.default_rng(seed)
        self.ctx, self.new = np.asarray(ctx), np.asarray(new)
        self.hq, self.hkv, self.d = hq, hkv, d
        self.q_dtype, self.kv_dtype = q_dtype, kv_dtype
        total = self.ctx + self.new
        pages = (total + 15) // 16
        self.indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.last = np.where(pages > 0, total - (pages - 1) * 16, 16).astype(np.int32)
        self.append = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.num_pages = int(self.indptr[-1]) + extra
        self.ids = rng.permutation(self.num_pages)[:self.indptr[-1]].astype(np.int32)
        self.T = int(self.append[-1])
        self.indices = torch.from_numpy(self.ids).to(device)
        x = rng.standard_normal((self.T, hq + 2 * hkv, d)) * 2.0 ** rng.uniform(-3, 3, (self.T, 1, 1))
        self.qkv = torch.from_numpy(x.astype(np.float32)).to(q_dtype).to(device)
        self.q, self.k, self.v = self.qkv.split([hq, hkv, hkv], 1)
        if kv_dtype == E4M3:
            codes = rng.integers(0, 256, (self.num_pages, 2, 16, hkv, d)).astype(np.uint8)
            self.kv = torch.from_numpy(codes).to(device).view(E4M3)
        else:
            kv = rng.standard_normal((self.num_pages, 2, 16, hkv, d)).astype(np.float32)
            self.kv = torch.from_numpy(kv).to(kv_dtype).to(device)

    def plan(self, fa, rotary=None, offset=None, **kw):
        return fa.plan_append(self.indptr, self.indices, self.last, self.append, self.hq,
                              self.hkv, self.d, 16, q_data_type=self.q_dtype,
                              kv_data_type=self.kv_dtype, rotary=rotary, position_offset=offset,
                              **kw)

    def places(self):
        """(request, row, page, slot, index in the request) of every new token."""
        out = []
        for i in range(len(self.ctx)):
            for j in range(self.new[i]):
                t = self.ctx[i] + j
                out.append((i, self.append[i] + j, int(self.ids[self.indptr[i] + t // 16]),
                            int(t % 16), int(t)))
        return out


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rotate(x, positions, rotary):
    """x [T, H, D] float64 rotated at positions [T]; the bound of its fp32 error."""
    y, slack = x.copy(), np.zeros_like(x)
    if rotary is None:
        return y, slack
    a = np.asarray(positions, np.float64)[:, None] * rotary.inv_freq
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    h = rotary.rotary_dim // 2
    i1 = 2 * np.arange(h) if rotary.interleaved else np.arange(h)
    i2 = i1 + (1 if rotary.interleaved else h)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    slack[..., i1] = slack[..., i2] = ROT * (np.abs(x[..., i1]) + np.abs(x[..., i2]))
    return y, slack


def positions_of(b, offset=None):
    off = np.zeros(len(b.ctx), np.int64) if offset is None else np.asarray(offset, np.int64)
    return np.array([off[i] + t for i, _, _, _, t in b.places()], np.int64)


def close(got, want, slack, dtype):
    bad = np.abs(got - want) > HALF[dtype] * np.abs(want) + slack * (1 + HALF[dtype]) + 1e-30
    if dtype == F16:  # subnormal steps
        bad &= np.abs(got - want) > 2.0 ** -25 + slack
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def code_close(got, want, slack):
    """Codes against want / scale, both in code units."""
    w = np.clip(want, -448, 448)
    bad = ~(np.abs(got - w) <= np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10) + slack)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def block_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s, 0 for 0."""
    s = np.zeros_like(amax)
    nz = amax > 0
    e = np.floor(np.log2(amax[nz])).astype(int) - 12
    p = 2.0 ** e
    for _ in range(8):
        p = np.where(amax[nz] > 448 * p, 2 * p, p)
    s[nz] = np.maximum(p, 2.0 ** -126)
    return s


LENGTHS = [([0, 5, 15, 16, 31, 0, 40, 7, 0, 100], [1, 0, 1, 1, 2, 0, 37, 9, 16, 1]),
           ([0], [1]), ([33], [70])]


# ---------------------------------------------------------------- native caches

@pytest.mark.gpu
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("rotary_dim,interleaved", [(0, False), (None, False), (None, True),
                                                    (16, False), (48, True), (32, False)])
@pytest.mark.parametrize("dtype,d,hq,hkv", [(F32, 64, 8, 8), (F32, 128, 3, 3), (BF16, 128, 32, 8),
                                            (BF16, 64, 10, 5), (F16, 128, 7, 1), (F16, 64, 16, 2),
                                            (BF16, 128, 34, 17)])
def test_native(lib, cuda, dtype, d, hq, hkv, rotary_dim, interleaved, lengths):
    b = Batch(*LENGTHS[lengths], hq, hkv, d, dtype, dtype, seed=d + hq + lengths)
    rd = d if rotary_dim is None else rotary_dim
    rot = lib.RotaryTable(rd, interleaved=interleaved) if rd else None
    p = b.plan(lib, rot)
    before = b.kv.clone()
    q = p.run(b.k, b.v, b.kv, q=b.q)
    torch.cuda.synchronize()
    assert p.check() == 0
    pos = positions_of(b)
    want, slack = rotate(f64(b.q), pos, rot)
    assert q.shape == b.q.shape and q.dtype == dtype and q.is_contiguous()
    close(f64(q), want, slack, dtype)
    k, kslack = rotate(f64(b.k), pos, rot)
    written = torch.zeros(b.num_pages, 16, dtype=torch.bool)
    for _, row, page, slot, _ in b.places():
        written[page, slot] = True
        close(f64(b.kv[page, 0, slot]), k[row], kslack[row], dtype)
        assert torch.equal(b.kv[page, 1, slot], b.v[row])
    keep = ~written.to(cuda)
    assert torch.equal(b.kv.transpose(1, 2)[keep], before.transpose(1, 2)[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1_000_000, 2_000_000_000, 2 ** 31 - 60])
@pytest.mark.parametrize("scale", [1.0, 0.125, 37.5, -1.0])
def test_far_positions(lib, cuda, offset, scale):
    """Angles keep their precision wherever a token stands: the reference's
    float64 angle is off by position * 2^-53 radians, 2.4e-7 at 2^31 (times the
    frequency), which joins the bound."""
    b = Batch([3, 20], [30, 2], 4, 2, 128, F32, F32, seed=5)
    freq = scale * 10000.0 ** (-2.0 * np.arange(64) / 128)
    rot = lib.RotaryTable(128, inv_freq=freq)
    p = b.plan(lib, rot, offset=[offset, offset // 3])
    q = p.run(b.k, b.v, b.kv, q=b.q)
    # the reduced angle in extended precision where the host has it
    pos = positions_of(b, [offset, offset // 3])
    two_pi = 6.283185307179586476925286766559
    ang = pos[:, None].astype(object)
    exact = np.empty((len(pos), 64))
    from fractions import Fraction
    tp = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    for i in range(len(pos)):
        for j in range(64):
            a = Fraction(int(ang[i, 0])) * Fraction(float(freq[j]))
            exact[i, j] = float(a - tp * (a // tp))
    del two_pi
    x = f64(b.q)
    c, s = np.cos(exact)[:, None], np.sin(exact)[:, None]
    want = np.concatenate([x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s], -1)
    slack = ROT * np.tile(np.abs(x[..., :64]) + np.abs(x[..., 64:]), 2)
    # the table's own frequencies: inv_freq / 2 pi to 2^-65 turns or the double's 2^-53
    # relative, whichever is larger, times the position
    extra = np.tile(2 * np.pi * pos[:, None] * 2.0 ** -63, (1, 64))[:, None]
    slack = slack + np.tile(extra, 2) * np.tile(np.abs(x[..., :64]) + np.abs(x[..., 64:]), 2)
    close(f64(q), want, slack, F32)


@pytest.mark.gpu
def test_in_place_stream_and_repeat(lib, cuda):
    """q rotated in place, on another stream, twice over the same slots."""
    b = Batch([0, 9], [21, 3], 8, 2, 128, BF16, BF16, seed=8)
    rot = lib.RotaryTable(128)
    p = b.plan(lib, rot)
    ref = p.run(b.k, b.v, b.kv, q=b.q)
    torch.cuda.synchronize()
    kv = b.kv.clone()
    q = b.q.contiguous()
    b.kv.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = p.run(b.k, b.v, b.kv, q=q, q_out=q)
    side.synchronize()
    assert out is q and torch.equal(q, ref)
    for _, _, page, slot, _ in b.places():
        assert torch.equal(b.kv[page, :, slot], kv[page, :, slot])
    assert p.run(b.k, b.v, b.kv) is None  # K and V alone


@pytest.mark.gpu
def test_graph_replay_with_new_inputs(lib, cuda):
    b = Batch([0, 9, 30], [1, 1, 1], 8, 2, 128, BF16, E4M3, seed=9)
    ks = torch.ones((b.num_pages, 2), device=cuda) * 2.0 ** -6
    vs = ks.clone()
    p = b.plan(lib, lib.RotaryTable(128))
    q = torch.empty_like(b.q.contiguous())
    kv0 = b.kv.clone()
    p.run_block_scales(b.k, b.v, b.kv, ks, vs, q=b.q, q_out=q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run_block_scales(b.k, b.v, b.kv, ks, vs, q=b.q, q_out=q)
    b.qkv.mul_(3.0)
    b.kv.view(torch.uint8).copy_(kv0.view(torch.uint8))
    ks.fill_(2.0 ** -6)
    vs.fill_(2.0 ** -6)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (q, b.kv.view(torch.uint8), ks, vs)]
    b.kv.view(torch.uint8).copy_(kv0.view(torch.uint8))
    ks.fill_(2.0 ** -6)
    vs.fill_(2.0 ** -6)
    p.run_block_scales(b.k, b.v, b.kv, ks, vs, q=b.q, q_out=q)
    torch.cuda.synchronize()
    for x, y in zip(got, (q, b.kv.view(torch.uint8), ks, vs)):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_nothing_to_append(lib, cuda):
    for ctx, new in (([], []), ([5, 0], [0, 0])):
        b = Batch(ctx, new, 8, 2, 64, BF16, BF16)
        before = b.kv.clone()
        q = b.plan(lib, lib.RotaryTable(64)).run(b.k, b.v, b.kv, q=b.q)
        torch.cuda.synchronize()
        assert q.shape == (0, 8, 64) and torch.equal(b.kv, before)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["native", "token", "block"])
def test_bad_page_ids_are_skipped(lib, cuda, mode):
    """A page id outside the cache is flagged, its tokens are not written, its
    q rows are; the other pages are written all the same."""
    b = Batch([0, 0, 20], [20, 3, 3], 8, 2, 128, BF16, BF16 if mode == "native" else E4M3, seed=3)
    bad = {1: b.num_pages, 2: -1}
    ids = b.ids.copy()
    for at, value in bad.items():
        ids[at] = value
    b.indices.copy_(torch.from_numpy(ids))
    shape = (b.num_pages, 2, 16) if mode == "token" else (b.num_pages, 2)
    ks, vs = (torch.full(shape, 0.5, device=cuda) for _ in range(2))
    before = b.kv.view(torch.uint8).clone()
    p = b.plan(lib, lib.RotaryTable(128))
    if mode == "native":
        q = p.run(b.k, b.v, b.kv, q=b.q)
    elif mode == "token":
        q = p.run_token_scales(b.k, b.v, b.kv, ks, vs, q=b.q)
    else:
        q = p.run_block_scales(b.k, b.v, b.kv, ks, vs, q=b.q)
    assert p.check() == 1 and p.check() == 0
    want, slack = rotate(f64(b.q), positions_of(b), lib.RotaryTable(128))
    close(f64(q), want, slack, BF16)
    after = b.kv.view(torch.uint8)
    good = {(page, slot) for i, _, page, slot, t in b.places()
            if int(b.indptr[i] + t // 16) not in bad}
    for page in range(b.num_pages):
        for slot in range(16):
            same = torch.equal(after[page, :, slot], before[page, :, slot])
            touched = mode == "block" and page in {x for x, _ in good}
            assert same == ((page, slot) not in good) or touched


# ---------------------------------------------------------------- E4M3 caches

@pytest.mark.gpu
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("dtype,d,hq,hkv", [(BF16, 128, 64, 8), (F16, 128, 5, 5), (BF16, 64, 6, 3),
                                            (F16, 64, 8, 1)])
@pytest.mark.parametrize("mode", ["tensor", "head", "token"])
def test_e4m3_given_and_token_scales(lib, cuda, mode, dtype, d, hq, hkv, lengths):
    b = Batch(*LENGTHS[lengths], hq, hkv, d, dtype, E4M3, seed=d + hq + lengths)
    rot = lib.RotaryTable(d, 500000.0)
    p = b.plan(lib, rot)
    before = b.kv.view(torch.uint8).clone()
    pos = positions_of(b)
    k, kslack = rotate(f64(b.k), pos, rot)
    v, vslack = f64(b.v), np.zeros((b.T, hkv, d))
    if mode == "tensor":
        q = p.run(b.k, b.v, b.kv, q=b.q, k_scale=0.03, v_scale=0.25)
        sk, sv = np.full((b.T, hkv), np.float32(0.03)), np.full((b.T, hkv), 0.25)
    elif mode == "head":
        hk = 0.01 * (1 + torch.arange(hkv, device=cuda, dtype=torch.float32))
        q = p.run_head_scales(b.k, b.v, b.kv, hk, 2 * hk, q=b.q)
        sk, sv = np.tile(f64(hk), (b.T, 1)), np.tile(2 * f64(hk), (b.T, 1))
    else:
        ks, vs = (torch.full((b.num_pages, hkv, 16), 7.0, device=cuda) for _ in range(2))
        q = p.run_token_scales(b.k, b.v, b.kv, ks, vs, q=b.q)
        sk, sv = np.empty((b.T, hkv)), np.empty((b.T, hkv))
        left = torch.ones(b.num_pages, 16, dtype=torch.bool)
        for _, row, page, slot, _ in b.places():
            sk[row], sv[row] = f64(ks[page, :, slot]), f64(vs[page, :, slot])
            left[page, slot] = False
        want = np.abs(k).max(-1) / 448
        # half a step of fp32 for the division, and the rotation's error
        assert (np.abs(sk - want) <= 2.0 ** -23 * want + kslack.max(-1) / 448).all()
        want = np.abs(v).max(-1) / 448
        assert (np.abs(sv - want) <= 2.0 ** -24 * want).all()
        for s in (ks, vs):
            assert (s.transpose(1, 2)[left.to(cuda)] == 7.0).all()
    want, slack = rotate(f64(b.q), pos, rot)
    close(f64(q), want, slack, dtype)
    after = b.kv.cpu()
    written = torch.zeros(b.num_pages, 16, dtype=torch.bool)
    for _, row, page, slot, _ in b.places():
        written[page, slot] = True
        for half, x, sl, s in ((0, k, kslack, sk), (1, v, vslack, sv)):
            w = x[row] / s[row][:, None]
            # the division by the scale in fp32: 2^-22 of the value with the
            # reciprocal's rounding
            code_close(f64(after[page, half, slot]), w,
                       sl[row] / s[row][:, None] * 1.1 + 2.0 ** -22 * np.abs(w))
    keep = ~written.to(cuda)
    assert torch.equal(b.kv.view(torch.uint8).transpose(1, 2)[keep], before.transpose(1, 2)[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("dtype,d,hq,hkv", [(BF16, 128, 64, 8), (F16, 128, 5, 5), (BF16, 64, 6, 3),
                                            (F16, 64, 8, 1), (BF16, 64, 33, 33)])
@pytest.mark.parametrize("spread", [0, 6, 30])
def test_block_scales(lib, cuda, spread, dtype, d, hq, hkv, lengths):
    """Scales and codes of continued and of new pages; spread: how far (log2)
    the pages' earlier scales lie from what the new tokens need."""
    b = Batch(*LENGTHS[lengths], hq, hkv, d, dtype, E4M3, seed=d + hq + lengths + spread)
    rng = np.random.default_rng(spread)
    rot = lib.RotaryTable(d)
    p = b.plan(lib, rot)
    old = [2.0 ** (-6 + np.rint(rng.uniform(-spread, spread, (b.num_pages, hkv)))) for _ in range(2)]
    old[0][rng.random(old[0].shape) < 0.1] = 0.0
    # without NaN codes among the earlier ones, which have no order
    raw = b.kv.view(torch.uint8)
    raw.copy_(torch.where((raw & 0x7f) == 0x7f, raw & 0x80, raw))
    before = b.kv.cpu().clone()
    ks, vs = (torch.from_numpy(s.astype(np.float32)).to(cuda) for s in old)
    q = p.run_block_scales(b.k, b.v, b.kv, ks, vs, q=b.q)
    torch.cuda.synchronize()
    assert p.check() == 0
    pos = positions_of(b)
    want, slack = rotate(f64(b.q), pos, rot)
    close(f64(q), want, slack, dtype)
    k, kslack = rotate(f64(b.k), pos, rot)
    data = ((k, kslack), (f64(b.v), np.zeros_like(k)))
    after, scales = b.kv.cpu(), (f64(ks), f64(vs))
    by_page = {}
    for _, row, page, slot, _ in b.places():
        by_page.setdefault(page, []).append((row, slot))
    for page in range(b.num_pages):
        if page not in by_page:
            assert torch.equal(after[page].view(torch.uint8), before[page].view(torch.uint8))
            for half in range(2):
                assert (scales[half][page] == old[half].astype(np.float32)[page]).all()
            continue
        rows, slots = (list(x) for x in zip(*by_page[page]))
        first = min(slots)
        for half, (x, sl) in enumerate(data):
            had = old[half][page] if first else np.zeros(hkv)
            got = scales[half][page]
            amax, near = np.abs(x[rows]).max((0, 2)), sl[rows].max((0, 2))
            lo, hi = (np.maximum(had, block_scale(np.maximum(amax + e, 0))) for e in (-near, near))
            assert ((got == lo) | (got == hi)).all()
            inv = np.where(got > 0, 1 / np.where(got > 0, got, 1), 0)
            for row, slot in zip(rows, slots):
                code_close(f64(after[page, half, slot]), x[row] * inv[:, None],
                           sl[row] * inv[:, None] * 1.1)
            # earlier codes: the nearest to the same values under the new
            # scale, bit for bit (torch's cast rounds to nearest even)
            ratio = np.where(got > had, had * inv, 1.0)
            moved = torch.from_numpy(f64(before[page, half, :first]) * ratio[None, :, None])
            assert torch.equal(after[page, half, :first].float(), moved.float().to(E4M3).float())
            end = max(slots) + 1
            assert torch.equal(after[page, half, end:].view(torch.uint8),
                               before[page, half, end:].view(torch.uint8))


@pytest.mark.gpu
def test_block_scales_token_by_token(lib, cuda):
    """A page filled one token at a time ends with the scale of one filled at
    once, and with the same codes but for those that passed through subnormals
    of a scale (each re-rounding is at most half a subnormal step of the scale
    it went to, and the scales at least double: together under one step)."""
    n = 40
    b = Batch([0, 0], [n, n // 2], 8, 4, 128, BF16, E4M3, seed=11)
    rot = lib.RotaryTable(128)
    ks, vs = (torch.full((b.num_pages, 4), 99.0, device=cuda) for _ in range(2))
    b.plan(lib, rot).run_block_scales(b.k, b.v, b.kv, ks, vs)
    kv1, ks1, vs1 = torch.zeros_like(b.kv.view(torch.uint8)).view(E4M3), ks * 0 + 99, vs * 0 + 99
    for t in range(n):
        rows = [i for i in range(2) if t < b.new[i]]
        total = np.array([min(t + 1, x) for x in b.new])
        pages = (total + 15) // 16
        # the request's page list up to now
        ids = np.concatenate([b.ids[b.indptr[i]:b.indptr[i] + pages[i]] for i in range(2)])
        indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        last = (total - (pages - 1) * 16).astype(np.int32)
        one = np.array([1 if t < x else 0 for x in b.new])
        p = lib.plan_append(indptr, torch.from_numpy(ids.astype(np.int32)).to(cuda), last,
                            np.concatenate([[0], np.cumsum(one)]).astype(np.int32), 8, 4, 128, 16,
                            q_data_type=BF16, kv_data_type=E4M3, rotary=rot)
        at = torch.tensor([int(b.append[i]) + t for i in rows], device=cuda)
        p.run_block_scales(b.k[at], b.v[at], kv1, ks1, vs1)
        torch.cuda.synchronize()
    for i in range(2):
        for pg in range((int(b.new[i]) + 15) // 16):
            page = int(b.ids[b.indptr[i] + pg])
            valid = min(16, int(b.new[i]) - 16 * pg)
            assert torch.equal(ks[page], ks1[page]) and torch.equal(vs[page], vs1[page])
            x, y = f64(b.kv[page, :, :valid]), f64(kv1[page, :, :valid])
            differ = x != y
            assert (np.abs(x - y) <= 2.0 ** -9)[differ].all()
            assert (np.abs(x)[differ] < 2.0 ** -6 + 2.0 ** -9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["tensor", "token", "block"])
def test_zeros_saturation_and_non_finite(lib, cuda, mode):
    b = Batch([0, 4], [3, 2], 2, 2, 64, BF16, E4M3, seed=2)
    x = torch.zeros((5, 2, 64), dtype=BF16, device=cuda)
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2], x[0, 0, 3] = float("inf"), float("nan"), 2.0, -float("inf")
    x[1, 0, 5] = -3.0e38
    x[1, 1, 5] = 1e-38  # below the smallest scale's codes
    x[3, 1] = 448.0     # 448 exactly: scale 1
    shape = (b.num_pages, 2, 16) if mode == "token" else (b.num_pages, 2)
    ks, vs = (torch.zeros(shape, device=cuda) for _ in range(2))
    p = b.plan(lib)
    if mode == "tensor":
        p.run(x, x, b.kv, k_scale=0.5, v_scale=0.5)
    else:
        getattr(p, f"run_{mode}_scales")(x, x, b.kv, ks, vs)
    torch.cuda.synchronize()
    for _, row, page, slot, _ in b.places():
        for half, sc in ((0, ks), (1, vs)):
            code = f64(b.kv[page, half, slot])
            if mode == "tensor":
                s = np.full(2, 0.5)
            else:
                s = f64(sc[page, :, slot] if mode == "token" else sc[page])
            val = code * s[:, None]
            w = f64(x[row])
            assert np.isnan(code[~np.isfinite(w)]).all()
            fin = np.isfinite(w)
            lim = np.clip(w, -448 * s[:, None], 448 * s[:, None])
            step = np.maximum(2.0 ** -4 * np.abs(lim), 2.0 ** -10 * s[:, None])
            assert (np.abs(val - lim) <= step * (1 + 2.0 ** -20))[fin].all()
            if mode == "token":
                assert ((s == 0) == (np.where(fin, np.abs(w), 0).max(-1) == 0)).all()
    if mode == "block":
        pg = int(b.ids[b.indptr[1]])
        assert float(ks[pg, 1]) == 1.0 and float(vs[pg, 1]) == 1.0
        assert float(ks[pg, 0]) == 0.0


# ---------------------------------------------------------------- as used: append, then decode

@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["native", "head", "token", "block"])
def test_append_then_decode(lib, cuda, mode):
    """Prompts, then decode steps, into one cache: what the steps attend to is
    what the oracle computes from the cache's own stored values and the rotated
    q; and those lie within rounding of the unquantised sequence."""
    hq, hkv, d = 16, 4, 128
    kvt = BF16 if mode == "native" else E4M3
    rot = lib.RotaryTable(d)
    prompts, steps = [1, 37, 16, 90], 3
    B = len(prompts)
    final = Batch([0] * B, [n + steps for n in prompts], hq, hkv, d, BF16, kvt, seed=21)
    final.kv.view(torch.uint8).fill_(0x7f)  # NaN in every slot not yet written
    shape = {"token": (final.num_pages, hkv, 16), "block": (final.num_pages, hkv)}.get(mode, (hkv,))
    ks, vs = (torch.full(shape, 0.05 if mode == "head" else float("nan"), device=cuda)
              for _ in range(2))

    def call(plan, rows):
        args = (final.k[rows], final.v[rows], final.kv)
        if mode == "native":
            return plan.run(*args, q=final.q[rows])
        return getattr(plan, f"run_{mode}_scales")(*args, ks, vs, q=final.q[rows])

    for step in range(steps + 1):
        total = np.array(prompts) + step
        new = np.array(prompts) if step == 0 else np.ones(B, int)
        pages = (total + 15) // 16
        ids = np.concatenate([final.ids[final.indptr[i]:final.indptr[i] + pages[i]]
                              for i in range(B)])
        indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        last = (total - (pages - 1) * 16).astype(np.int32)
        dev_ids = torch.from_numpy(ids).to(cuda)
        rows = torch.from_numpy(np.concatenate(
            [final.append[i] + np.arange(total[i] - new[i], total[i]) for i in range(B)])).to(cuda)
        ap = lib.plan_append(indptr, dev_ids, last, np.concatenate([[0], np.cumsum(new)]), hq, hkv,
                             d, 16, q_data_type=BF16, kv_data_type=kvt, rotary=rot)
        q = call(ap, rows)
        if step == 0:
            continue
        dp = lib.plan(indptr, dev_ids, last, hq, hkv, d, 16, q_data_type=BF16, kv_data_type=kvt)
        if mode == "native":
            o, lse = dp.run(q, final.kv)
        else:
            o, lse = getattr(dp, f"run_{mode}_scales")(q, final.kv, ks, vs)
        torch.cuda.synchronize()
        assert ap.check() == 0 and dp.check() == 0
        kv = final.kv.float()
        if mode == "head":
            kv = kv * 0.05
        elif mode == "token":
            s = torch.stack([ks, vs], 1).permute(0, 1, 3, 2)[..., None]
            kv = kv * s
        elif mode == "block":
            kv = kv * torch.stack([ks, vs], 1)[:, :, None, :, None]
        qb, qc = as_bits(q)
        ref_o, ref_lse = oracle.batch_decode(qb, qc, kv.cpu().numpy(), oracle.F32, indptr, ids,
                                             last, hq, hkv, d, 16)
        vmax = float(kv[:, 1].nan_to_num().abs().max())
        assert np.abs(f64(o) - ref_o).max() <= 2.0 ** -8 * np.abs(ref_o).max() + 2.0 ** -8 * vmax
        assert np.abs(f64(lse) - ref_lse).max() <= 2e-3


# ---------------------------------------------------------------- refusals

def host_plan(lib, *, indptr=(0, 1), last=(3,), append=(0, 2), offset=None, hq=8, hkv=2, d=128,
              page=16, q=1, kv=1, freq=None, rotary=0, ws=256, ws_bytes=1 << 20, indices=256,
              batch=None):
    """fa_append_plan with addresses that no refused call touches."""
    L = lib.library()
    arr = lambda v: np.array(v, np.int32)  # noqa: E731
    a, l, p = arr(indptr), arr(last), arr(append)
    o = None if offset is None else arr(offset)
    f = None if freq is None else np.array(freq, np.float64)
    out = ctypes.c_void_p()
    rc = L.fa_append_plan(a.ctypes.data, indices, l.ctypes.data, p.ctypes.data,
                          o.ctypes.data if o is not None else None,
                          len(a) - 1 if batch is None else batch, hq, hkv, d, page, q, kv,
                          f.ctypes.data if f is not None else None, rotary, 0, ws, ws_bytes, None,
                          ctypes.byref(out))
    assert not out.value
    return rc


def test_plan_refusals(lib):
    """Each refused on the host, before any CUDA call."""
    invalid, unsupported, small = -1, -2, -3
    for kw, rc in [
            (dict(indptr=(0, 0), append=(0, 1)), invalid),         # no page to append to
            (dict(append=(0, 4)), invalid),                        # more new tokens than tokens
            (dict(append=(1, 2)), invalid), (dict(indptr=(1, 2)), invalid),
            (dict(append=(0, -1)), invalid), (dict(indptr=(0, -1)), invalid),
            (dict(last=(0,)), invalid), (dict(last=(17,)), invalid),
            (dict(offset=(-1,)), invalid), (dict(offset=(2 ** 31 - 3,)), invalid),
            (dict(hq=7), invalid), (dict(hkv=0), invalid), (dict(ws=None), invalid),
            (dict(ws=128), invalid), (dict(indices=None), invalid), (dict(batch=-1), invalid),
            (dict(rotary=144, freq=[1.0] * 72), invalid), (dict(rotary=16), invalid),
            (dict(rotary=16, freq=[float("nan")] * 8), invalid),
            (dict(rotary=16, freq=[float("inf")] * 8), invalid),
            (dict(rotary=16, freq=[-1e10] * 8), invalid),
            (dict(rotary=8, freq=[1.0] * 4), unsupported), (dict(d=96), unsupported),
            (dict(page=32, last=(32,)), unsupported), (dict(q=0, kv=1), unsupported),
            (dict(q=0, kv=3), unsupported), (dict(q=1, kv=2), unsupported),
            (dict(q=3, kv=3), unsupported), (dict(q=9), unsupported),
            (dict(ws_bytes=256), small)]:
        assert host_plan(lib, **kw) == rc, kw


def test_null_arguments(lib):
    L = lib.library()
    assert L.fa_append_plan_destroy(None) == 0
    assert L.fa_append_run(None, None, None, None, None, None, 1, 1.0, 1.0, None) == -1
    for name in ("head", "token", "block"):
        f = getattr(L, f"fa_append_run_{name}_scales")
        assert f(None, None, None, None, None, None, 1, None, None, None) == -1
    assert L.fa_append_check(None, None, None) == -1
    assert L.fa_decode_run_block_scales(None, None, None, 1, 0.0, None, None, None, None, None) == -1


def test_workspace_size(lib):
    assert lib.append_workspace_size(0, 0) > 0
    assert lib.append_workspace_size(64, 100_000) >= 16 * (100_000 // 16 + 64)
    for bad in ((-1, 5), (1, -5), (1, 2 ** 31)):
        with pytest.raises(ValueError):
            lib.append_workspace_size(*bad)


def test_rotary_table(lib):
    t = lib.RotaryTable(32, 500000.0)
    np.testing.assert_allclose(t.inv_freq, 500000.0 ** (-np.arange(16) / 16.0), rtol=1e-15)
    for bad in (0, 8, 20, -16):
        with pytest.raises(ValueError):
            lib.RotaryTable(bad)
    with pytest.raises(ValueError):
        lib.RotaryTable(32, inv_freq=np.ones(32))
    with pytest.raises(ValueError):
        lib.RotaryTable(32, inv_freq=[float("nan")] * 16)


@pytest.mark.gpu
def test_run_refusals(lib, cuda):
    b = Batch([0, 5], [4, 2], 8, 2, 128, BF16, E4M3, seed=1)
    p = b.plan(lib, lib.RotaryTable(128))
    ks = torch.ones((b.num_pages, 2), device=cuda)
    kt = torch.ones((b.num_pages, 2, 16), device=cuda)
    before = b.kv.view(torch.uint8).clone()
    odd = torch.empty(b.k.numel() + 8, dtype=BF16, device=cuda)[4:b.k.numel() + 4].view(b.k.shape)
    for bad in (lambda: p.run(b.k.float(), b.v, b.kv), lambda: p.run(b.k[:-1], b.v, b.kv),
                lambda: p.run(b.k, b.v, b.kv.float()), lambda: p.run(b.k, b.v, b.kv[:, :, ::2]),
                lambda: p.run(b.k.cpu(), b.v, b.kv), lambda: p.run(odd, b.v, b.kv),
                lambda: p.run(b.k.transpose(1, 2).contiguous().transpose(1, 2), b.v, b.kv),
                lambda: p.run(b.k, b.v, b.kv, k_scale=0.0),
                lambda: p.run(b.k, b.v, b.kv, v_scale=-1.0),
                lambda: p.run(b.k, b.v, b.kv, k_scale=1e-40),
                lambda: p.run(b.k, b.v, b.kv, v_scale=float("inf")),
                lambda: p.run(b.k, b.v, b.kv, k_scale=float("nan")),
                lambda: p.run(b.k, b.v, b.kv, q=b.q, q_out=b.q),
                lambda: p.run(b.k, b.v, b.kv, q_out=b.q.contiguous()),
                lambda: p.run_block_scales(b.k, b.v, b.kv, kt, kt),
                lambda: p.run_block_scales(b.k, b.v, b.kv, ks, ks.double()),
                lambda: p.run_block_scales(b.k, b.v, b.kv, ks, ks.cpu()),
                lambda: p.run_token_scales(b.k, b.v, b.kv, ks, ks),
                lambda: p.run_head_scales(b.k, b.v, b.kv, ks, ks)):
        with pytest.raises((ValueError, TypeError, lib.FaError)):
            bad()
    torch.cuda.synchronize()
    assert torch.equal(b.kv.view(torch.uint8), before)
    with pytest.raises(ValueError):
        b.plan(lib, workspace=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(lib.FaError):
        b.plan(lib, workspace=torch.empty(16, dtype=torch.uint8, device=cuda))
    n = Batch([0], [4], 8, 2, 128, BF16, BF16)
    pn = n.plan(lib)
    s = torch.ones((n.num_pages, 2), device=cuda)
    for bad in (lambda: pn.run(n.k, n.v, n.kv, k_scale=0.5),
                lambda: pn.run_block_scales(n.k, n.v, n.kv, s, s)):
        with pytest.raises(lib.FaError):
            bad()


@pytest.mark.gpu
def test_another_current_device_is_refused(lib, cuda, monkeypatch):
    """Index tensors and workspaces of a device that is not the current one."""
    b = Batch([0], [4], 8, 2, 128, BF16, BF16)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=cuda)
    other = torch.cuda.current_device() + 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: other)
    for kw in ({}, {"workspace": ws}):
        with pytest.raises(ValueError):
            b.plan(lib, **kw)


@pytest.mark.gpu
def test_continued_page_without_a_scale(lib, cuda):
    """A page that is continued although nothing wrote its scale (NaN) takes the
    scale its new tokens need."""
    b = Batch([5], [3], 2, 2, 64, BF16, E4M3, seed=4)
    ks, vs = (torch.full((b.num_pages, 2), float("nan"), device=cuda) for _ in range(2))
    b.plan(lib).run_block_scales(b.k, b.v, b.kv, ks, vs)
    page = int(b.ids[0])
    want = block_scale(np.abs(f64(b.k)).max((0, 2)))
    assert np.array_equal(f64(ks[page]), want)
    assert torch.isnan(ks[[i for i in range(b.num_pages) if i != page]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["native", "block"])
def test_large_cache(lib, cuda, mode):
    """Pages whose elements lie beyond 2^31 from the cache's start, and beyond
    2^32 bytes."""
    hkv, d = 8, 128
    pages = (1 << 31) // (2 * 16 * hkv * d) + 70000   # 4.5 GB of E4M3, 9 GB of bf16
    kvt = BF16 if mode == "native" else E4M3
    es = 2 if mode == "native" else 1
    raw = torch.zeros(pages * 2 * 16 * hkv * d * es, dtype=torch.uint8, device=cuda)
    kv = raw.view(kvt).view(pages, 2, 16, hkv, d)
    ids = torch.tensor([pages - 1, 3, pages - 65000], dtype=torch.int32, device=cuda)
    k = torch.randn((40, hkv, d), device=cuda).to(BF16)
    v = torch.randn((40, hkv, d), device=cuda).to(BF16)
    p = lib.plan_append([0, 3], ids, [8], [0, 40], 8, hkv, d, 16, q_data_type=BF16,
                        kv_data_type=kvt)
    if mode == "native":
        p.run(k, v, kv)
        got = kv[ids.long()].transpose(1, 2).reshape(48, 2, hkv, d)[:40]
        assert torch.equal(got[:, 0], k) and torch.equal(got[:, 1], v)
    else:
        ks, vs = (torch.zeros((pages, hkv), device=cuda) for _ in range(2))
        p.run_block_scales(k, v, kv, ks, vs)
        s = torch.stack([ks, vs], 1)[ids.long()][:, :, None, :, None]
        got = (kv[ids.long()].float() * s).transpose(1, 2).reshape(48, 2, hkv, d)[:40]
        step = s.amax((0, 1, 2)) * 2.0 ** -10
        for x, y in ((got[:, 0], k.float()), (got[:, 1], v.float())):
            assert ((x - y).abs() <= torch.maximum(2.0 ** -4 * y.abs(), step)).all()
        dp = lib.plan([0, 3], ids, [8], 8, hkv, d, 16, q_data_type=BF16, kv_data_type=kvt)
        q = torch.randn((1, 8, d), device=cuda).to(BF16)
        o, _ = dp.run_block_scales(q, kv, ks, vs)
        w = torch.softmax(torch.einsum("hd,thd->ht", q[0].double(), got[:, 0].double()) / d ** 0.5, -1)
        ref = torch.einsum("ht,thd->hd", w, got[:, 1].double())
        # bf16's half step, and 3 * 2^-11 + 2e-4 of the weights' values (see the
        # block-scale tests)
        mag = torch.einsum("ht,thd->hd", w, got[:, 1].double().abs())
        assert ((o[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2e-3 * mag).all()
    assert p.check() == 0
    assert not raw[: 3 * 2 * 16 * hkv * d * es].any()

"""Attention of packed query rows (plan_prefill) against the definition in 64 bits,
its planner on the CPU, and its refusals.

Tolerances.  The weights enter P V rounded to the type of q by half a step (HALF:
bf16 2^-8, f16 2^-11), the output once more; so |o - exact| <= HALF (sum_t w_t |v_t|
+ |o|) with w the softmax weights.  An f16 weight below 2^-14 of the reference is
subnormal, off by 2^-25 of it at most: 2^-25 sum_t |v_t| more.  A logit is a sum of D
exact products in fp32, in the tensor cores' order: its error is held to
D 2^-23 times the sum of the products' magnitudes (2^-24 an addition, twice that where
additions truncate), plus 2^-21 |logit| for the scaling, the exponential (2^-22)
and the sum; that moves every weight by twice its value relative (numerator and
denominator), and lse once.  An E4M3 cache's codes are exact in bf16 and K's scales
multiply the logits; V's elements under a scale per token or block that is no power of
two are rounded: HALF sum_t w_t |v_t| more.
"""
import ctypes

import numpy as np
import pytest
import torch

E4M3 = torch.float8_e4m3fn
BF16, F16 = torch.bfloat16, torch.float16
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}


class Batch:
    """Requests of ctx[i] + new[i] tokens, the last new[i] with query rows."""

    def __init__(self, ctx, new, hq, hkv, d, q_dtype=BF16, kv_dtype=None, seed=0, extra=3,
                 garbage=float("nan"), spread=1.0):
        rng = np.random.default_rng(seed)
        self.ctx, self.new = np.asarray(ctx, np.int64), np.asarray(new, np.int64)
        self.hq, self.hkv, self.d = hq, hkv, d
        self.q_dtype, self.kv_dtype = q_dtype, kv_dtype or q_dtype
        self.total = self.ctx + self.new
        pages = (self.total + 15) // 16
        self.indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.last = np.where(pages > 0, self.total - (pages - 1) * 16, 16).astype(np.int32)
        self.qo = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.num_pages = int(self.indptr[-1]) + extra
        self.ids = rng.permutation(self.num_pages)[:self.indptr[-1]].astype(np.int32)
        self.T = int(self.qo[-1])
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.indices = torch.from_numpy(self.ids).cuda()
        self.q = (torch.randn((self.T, hq, d), generator=g, device="cuda") * spread).to(q_dtype)
        kv = torch.randn((self.num_pages, 2, 16, hkv, d), generator=g, device="cuda")
        if self.kv_dtype == E4M3:
            kv = kv * 8
        self.kv = kv.to(self.kv_dtype)
        # what unused slots and pages hold is ignored
        used = np.zeros((self.num_pages, 16), bool)
        for i, n in enumerate(self.total):
            t = np.arange(n)
            used[self.ids[self.indptr[i] + t // 16], t % 16] = True
        unused = torch.from_numpy(~used).cuda()[:, None].expand(-1, 2, -1)
        raw = self.kv.view(torch.uint8) if self.kv_dtype == E4M3 else self.kv
        raw[unused] = 127 if self.kv_dtype == E4M3 else garbage
        self.scales = None

    def plan(self, fa, **kw):
        return fa.plan_prefill(self.indptr, self.indices, self.last, self.qo, self.hq, self.hkv,
                               self.d, 16, q_data_type=self.q_dtype, kv_data_type=self.kv_dtype,
                               **kw)

    def check(self, o, lse, scale_of=None, inexact=False, sm_scale=None, rows=None):
        """o and lse against the definition; scale_of(half, pages, slots): [tokens,
        hkv] factors of the elements; inexact: V's elements rounded to bf16."""
        half, d, G = HALF[self.q_dtype], self.d, self.hq // self.hkv
        sm = d ** -0.5 if sm_scale is None else sm_scale
        kv = self.kv.double()
        for i in range(len(self.total)):
            n, L = int(self.new[i]), int(self.total[i])
            if n == 0:
                continue
            t = torch.arange(L, device="cuda")
            page = self.indices[self.indptr[i]:self.indptr[i + 1]].long()[t // 16]
            k, v = kv[page, 0, t % 16], kv[page, 1, t % 16]
            if scale_of is not None:
                k, v = k * scale_of(0, page, t % 16)[..., None], v * scale_of(1, page, t % 16)[..., None]
            a = int(self.qo[i])
            pick = np.arange(n) if rows is None or n <= rows else np.unique(
                np.concatenate([[0, n - 1], np.random.default_rng(0).integers(0, n, rows)]))
            pick_t = torch.from_numpy(pick).cuda()
            q = self.q[a + pick_t].double()
            seen = t[None, :] <= (L - n + pick_t)[:, None]
            for h in range(self.hq):
                kh, vh = k[:, h // G], v[:, h // G]
                s = (q[:, h] @ kh.T * sm).masked_fill(~seen, -float("inf"))
                size = (q[:, h].abs() @ kh.abs().T * sm).masked_fill(~seen, 0).amax(-1)
                ref = torch.logsumexp(s, -1)
                w = (s - ref[:, None]).exp()
                want, mag = w @ vh, w @ vh.abs()
                err = size * d * 2.0 ** -23 + 2.0 ** -21 * (1 + size)
                bound = (half * (2 if inexact else 1) + 2 * err)[:, None] * mag + half * want.abs()
                bound = bound * 1.001 + 1e-30
                if self.q_dtype == F16:
                    bound += 2.0 ** -25 * ((seen.double() @ vh.abs()) + 1)
                got = o[a + pick_t, h].double()
                bad = ~((got - want).abs() <= bound)
                assert not bad.any(), (i, h, bad.nonzero()[:4], got[bad][:4], want[bad][:4], bound[bad][:4])
                if lse is not None:
                    bad = ~((lse[a + pick_t, h].double() - ref).abs() <= err + 2.0 ** -22 * ref.abs())
                    assert not bad.any(), (i, h, bad.nonzero()[:4], lse[a + pick_t, h][bad][:4], ref[bad][:4])


LENGTHS = [
    ([0, 5, 15, 16, 0, 31, 0, 100, 250], [1, 0, 1, 17, 0, 2, 37, 29, 7]),
    ([0], [1]), ([0], [128]), ([0], [129]), ([0], [300]), ([513], [64]), ([1000, 127], [1, 1]),
    ([2000, 0, 1], [33, 256, 255]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("dtype,d,hq,hkv", [
    (BF16, 128, 32, 8), (BF16, 128, 8, 1), (F16, 128, 3, 3), (F16, 64, 10, 5), (BF16, 64, 8, 2),
    (BF16, 128, 6, 3), (F16, 64, 8, 1), (BF16, 64, 1, 1)])
def test_native(lib, cuda, dtype, d, hq, hkv, lengths):
    b = Batch(*LENGTHS[lengths], hq, hkv, d, dtype, seed=lengths)
    p = b.plan(lib)
    o, lse = p.run(b.q, b.kv)
    assert p.check() == 0
    b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv,dtype", [(128, 32, 8, BF16), (64, 4, 4, F16)])
def test_long(lib, cuda, d, hq, hkv, dtype):
    """Rows of several items a CTA, contexts of hundreds of tiles; rows picked."""
    b = Batch([0, 9000, 31, 4000], [5000, 1700, 2900, 1], hq, hkv, d, dtype, seed=3)
    p = b.plan(lib)
    o, lse = p.run(b.q, b.kv)
    assert p.check() == 0
    b.check(o, lse, rows=40)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,ctx,new", [(8, 1, [30000], [1]), (4, 4, [70000], [3]),
                                            (32, 8, [9000, 20, 12000], [5, 4, 66])])
def test_split_keys(lib, cuda, hq, hkv, ctx, new):
    """Few rows over long contexts: their keys are split over SMs and folded."""
    b = Batch(ctx, new, hq, hkv, 128, seed=5)
    p = b.plan(lib)
    o, lse = p.run(b.q, b.kv)
    again, _ = p.run(b.q, b.kv)
    assert p.check() == 0 and torch.equal(o, again)
    b.check(o, lse)


@pytest.mark.gpu
def test_logits_that_grow(lib, cuda):
    """Maxima that rise tile after tile (the rescaled path), and by leaps."""
    for step in (0.02, 1.0):
        b = Batch([700], [90], 4, 1, 128, seed=6)
        t = torch.arange(790, device=cuda)
        page = b.indices.long()[t // 16]
        u = torch.randn(128, device=cuda)
        u /= u.norm()
        b.kv[page, 0, t % 16, 0] = (u[None] * (t[:, None] * step)).to(BF16)
        b.q[:] = (u * 11.3).to(BF16)
        p = b.plan(lib)
        o, lse = p.run(b.q, b.kv)
        b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", ["tensor", "head", "token", "block", "block_any"])
def test_e4m3(lib, cuda, mode, d):
    b = Batch([0, 40, 300, 1000], [70, 1, 130, 33], 16, 4, d, BF16, E4M3, seed=7)
    p = b.plan(lib)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    if mode == "tensor":
        o, lse = p.run(b.q, b.kv, k_scale=0.11, v_scale=0.3)
        of = lambda half, page, slot: torch.full((len(page), 4), (0.11, 0.3)[half],  # noqa: E731
                                                 dtype=torch.float64, device="cuda")
        # the call takes its scales in fp32: 2^-24 of them
        return b.check(o, lse, of)
    if mode == "head":
        s = [rand(4) * 0.2 + 0.01, rand(4) * 0.2 + 0.01]
        o, lse = p.run_head_scales(b.q, b.kv, *s)
        return b.check(o, lse, lambda half, page, slot: s[half].double().expand(len(page), 4))
    if mode == "token":
        s = [rand(b.num_pages, 4, 16) * 0.2 + 0.001 for _ in range(2)]
        o, lse = p.run_token_scales(b.q, b.kv, *s)
        return b.check(o, lse, lambda half, page, slot: s[half].double()[page, :, slot], True)
    if mode == "block":
        s = [torch.exp2(torch.floor(rand(b.num_pages, 4) * 9) - 9) for _ in range(2)]
    else:
        s = [rand(b.num_pages, 4) * 0.2 + 0.001 for _ in range(2)]
    o, lse = p.run_block_scales(b.q, b.kv, *s)
    assert p.check() == 0
    b.check(o, lse, lambda half, page, slot: s[half].double()[page], mode == "block_any")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_scales_behind_the_last_token_are_ignored(lib, cuda, d):
    b = Batch([0, 40, 300], [70, 1, 130], 16, 4, d, BF16, E4M3, seed=9)
    g = torch.Generator(device="cuda").manual_seed(2)
    s = [torch.rand((b.num_pages, 4, 16), generator=g, device="cuda") * 0.2 + 0.001 for _ in range(2)]
    unused = (b.kv.view(torch.uint8)[:, 0, :, :, 0] == 127).transpose(1, 2)
    for x in s:
        x[unused] = float("nan")
    o, lse = b.plan(lib).run_token_scales(b.q, b.kv, *s)
    b.check(o, lse, lambda half, page, slot: s[half].double()[page, :, slot], True)


@pytest.mark.gpu
def test_scales_of_zero(lib, cuda):
    """A scale of 0: all logits equal (K), all values 0 (V)."""
    b = Batch([20], [30], 4, 1, 128, BF16, E4M3, seed=8)
    p = b.plan(lib)
    o, lse = p.run(b.q, b.kv, k_scale=0.0)
    seen = 21 + torch.arange(30, device=cuda)
    torch.testing.assert_close(lse, seen.float().log()[:, None].expand(-1, 4), rtol=1e-6, atol=0)
    z = torch.zeros(1, device=cuda)
    o, lse2 = p.run_head_scales(b.q, b.kv, z, z)
    assert torch.equal(lse, lse2) and not o.any()


@pytest.mark.gpu
def test_matches_the_ragged_decode_plan(lib, cuda):
    """The same rows through plan_ragged_q.  Its denominator is the sum of the weights
    as rounded to bf16 (half a step, 2^-8 of each), so its lse may be ln(1 - 2^-8)
    = -2^-8 (1 + 2^-9 + ...) off, and its o twice the weights' rounding."""
    b = Batch([100, 40, 999], [4, 1, 3], 32, 8, 128, seed=9)
    o, lse = b.plan(lib).run(b.q, b.kv)
    r = lib.plan_ragged_q(b.indptr, b.indices, b.last, b.qo, 32, 8, 128, 16)
    o2, lse2 = r.run(b.q, b.kv)
    b.check(o, lse)
    b.check(o2, None, inexact=True)
    assert ((lse - lse2).abs() <= 2.0 ** -8 * 1.01).all()


@pytest.mark.gpu
def test_strided_rows_given_outputs_and_scale(lib, cuda):
    """q as a slice of a fused projection; outputs of the caller's; no lse."""
    b = Batch([0, 9], [70, 200], 16, 4, 128, seed=10)
    fused = torch.full((b.T, 24, 128), float("nan"), dtype=BF16, device=cuda)
    fused[:, 3:19] = b.q
    p = b.plan(lib)
    o, lse = p.run(b.q, b.kv, sm_scale=0.2)
    out = torch.empty_like(o)
    got = torch.empty_like(lse)
    a, l = p.run(fused[:, 3:19], b.kv, sm_scale=0.2, out=out, lse=got)
    assert a is out and l is got and torch.equal(out, o) and torch.equal(got, lse)
    by_head = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    a, l = p.run(by_head, b.kv, sm_scale=0.2, return_lse=False)
    assert l is None and torch.equal(a, o)
    b.check(o, lse, sm_scale=0.2)


@pytest.mark.gpu
def test_rows_of_others_stay(lib, cuda):
    """Rows behind the batch's last are not written."""
    b = Batch([3, 60], [100, 30], 8, 2, 128, seed=11)
    out = torch.full((b.T + 40, 8, 128), 7.0, dtype=BF16, device=cuda)
    lse = torch.full((b.T + 40, 8), 7.0, device=cuda)
    o, l = b.plan(lib).run(b.q, b.kv, out=out, lse=lse)
    b.check(out[:b.T], lse[:b.T])
    assert (out[b.T:] == 7).all() and (lse[b.T:] == 7).all()


@pytest.mark.gpu
def test_stream_and_graph(lib, cuda):
    b = Batch([50, 3000], [129, 5], 8, 2, 128, seed=12)
    p = b.plan(lib)
    o, lse = p.run(b.q, b.kv)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = p.run(b.q, b.kv, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    out, l = torch.empty_like(o), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(b.q, b.kv, out=out, lse=l)
    b.q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    b.check(out, l)


@pytest.mark.gpu
def test_two_plans_on_two_streams(lib, cuda):
    """Runs in flight together, each with a plan (and workspace) of its own; outputs and
    workspaces made for those streams."""
    b = [Batch([9000, 40], [5, 300], 8, 2, 128, seed=20), Batch([0, 7000], [700, 3], 8, 2, 128, seed=21)]
    want = [x.plan(lib).run(x.q, x.kv) for x in b]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    plans = [x.plan(lib, stream=st) for x, st in zip(b, streams)]
    got = []
    for _ in range(5):
        got.append([p.run(x.q, x.kv, stream=st) for x, p, st in zip(b, plans, streams)])
    torch.cuda.synchronize()
    for pair in got:
        for (o, lse), (ow, lw) in zip(pair, want):
            assert torch.equal(o, ow) and torch.equal(lse, lw)


@pytest.mark.gpu
def test_bad_page_ids_read_zeros(lib, cuda):
    b = Batch([0, 200], [40, 150], 8, 2, 128, seed=13)
    good, _ = b.plan(lib).run(b.q, b.kv)
    for bad in (-1, b.num_pages, 2 ** 31 - 1):
        ids = b.indices.clone()
        ids[int(b.indptr[1]) + 3] = bad
        kept, b.indices = b.indices, ids
        p = b.plan(lib)
        o, lse = p.run(b.q, b.kv)
        assert p.check() == 1 and p.check() == 0
        b.indices = kept
        assert torch.equal(o[:40], good[:40]) and torch.isfinite(o).all()
        # as a page of zeros
        at, z = int(b.ids[b.indptr[1] + 3]), b.kv.clone()
        z[at] = 0
        want, _ = b.plan(lib).run(b.q, z)
        assert torch.equal(o, want)


@pytest.mark.gpu
def test_no_rows(lib, cuda):
    for ctx, new in (([], []), ([5, 0], [0, 0])):
        b = Batch(ctx, new, 8, 2, 64)
        o, lse = b.plan(lib).run(b.q, b.kv)
        assert o.shape == (0, 8, 64) and lse.shape == (0, 8)


@pytest.mark.gpu
def test_shared_pages(lib, cuda):
    """Two requests over the same prefix pages."""
    b = Batch([64, 64], [20, 9], 8, 2, 128, seed=14)
    b.ids[b.indptr[1]:b.indptr[1] + 4] = b.ids[:4]
    b.indices = torch.from_numpy(b.ids).cuda()
    o, lse = b.plan(lib).run(b.q, b.kv)
    b.check(o, lse)


@pytest.mark.gpu
def test_infinite_logits_are_nan_as_by_definition(lib, cuda):
    b = Batch([0], [40], 2, 2, 64, garbage=0.0)
    b.kv[b.indices.long()[0], 0, 5, 0, 0] = float("inf")
    o, lse = b.plan(lib).run(b.q, b.kv)
    pos = b.q[:, 0, 0] > 0
    row = torch.arange(40, device=cuda)
    assert torch.isnan(o[(row >= 5) & pos, 0]).all() and torch.isfinite(o[row < 5]).all()
    assert torch.isfinite(o[:, 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,d,hq,hkv,ctx,new", [
    (BF16, 128, 8, 2, 40, 90), (F16, 64, 3, 3, 0, 300), (BF16, 64, 8, 1, 200, 60),
    (BF16, 128, 4, 4, 20000, 40)])  # (the last: keys split over SMs)
def test_values_that_a_row_does_not_see(lib, cuda, dtype, d, hq, hkv, ctx, new, value):
    """V of one token of the prompt is not finite: rows before it have their finite
    results, rows from it on have none in that dim.  K not finite: likewise."""
    b = Batch([ctx], [new], hq, hkv, d, dtype, seed=15)
    clean, lse = b.plan(lib).run(b.q, b.kv)
    at = new // 2
    page, slot = int(b.indices[(ctx + at) // 16]), (ctx + at) % 16
    kv = b.kv.clone()
    kv[page, 1, slot, 0, 5] = value
    p = b.plan(lib)
    o, l = p.run(b.q, kv)
    assert p.check() == 0 and torch.equal(l, lse)
    G = hq // hkv
    assert not torch.isfinite(o[at:, :G, 5]).any()
    o[at:, :G, 5] = clean[at:, :G, 5]
    b.check(o, l, rows=30)
    assert torch.equal(o[at:], clean[at:]) and torch.equal(o[:, G:], clean[:, G:])
    kv = b.kv.clone()
    kv[page, 0, slot, 0, 5] = value
    o, l = p.run(b.q, kv)
    assert torch.equal(o[:at], clean[:at]) and torch.equal(l[:at], lse[:at])


# ---------------------------------------------------------------- the planner (CPU)

def lay(total):
    pages = (np.asarray(total) + 15) // 16
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    return indptr, np.where(pages > 0, total - (pages - 1) * 16, 16).astype(np.int32)


@pytest.mark.parametrize("seed", range(30))
def test_work_list_covers_every_row_and_tile_once(lib, seed):
    rng = np.random.default_rng(seed)
    B, group, heads = int(rng.integers(0, 20)), int(rng.choice([1, 2, 4, 8])), int(rng.integers(1, 9))
    total = rng.integers(0, [50, 700, 9000, 60000][seed % 4], B)
    new = np.minimum(rng.integers(0, [2, 40, 700, 9000][seed // 4 % 4], B), total)
    indptr, last = lay(total)
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ctas = int(rng.choice([1, 7, 152]))
    offsets, items, merge, slots = lib.plan_prefill_host(indptr, last, qo, group, heads, ctas)
    assert len(offsets) - 1 <= ctas and offsets[0] == 0 and offsets[-1] == len(items)
    assert (np.diff(offsets) > 0).all()
    step, want, got = 256 // group, {}, {}
    for i in range(B):
        for t in range(0, new[i], step):
            n = min(step, new[i] - t)
            tiles = -(-(total[i] - new[i] + t + n) // 128)
            for h in range(heads):
                want[(qo[i] + t, n, total[i] - new[i] + t, indptr[i], h)] = tiles
    used = np.zeros(slots, int)
    for row0, n, pos0, entry, t0, t1, slot, h in items.tolist():
        assert t0 < t1 and (slot >= 0 or t0 == 0)
        got.setdefault((row0, n, pos0, entry, h), []).append((t0, t1, slot))
        if slot >= 0:
            used[slot] += 1
    assert (used == 1).all() and set(got) == set(want)
    units = {(r, n, h): (s, k) for r, n, s, k, h, _, _, _ in merge.tolist()}
    assert len(units) == len(merge)
    for key, pieces in got.items():
        pieces.sort()
        assert [p[0] for p in pieces] == [0] + [p[1] for p in pieces[:-1]]
        assert pieces[-1][1] == want[key]
        unit = units.pop((key[0], key[1], key[4]), None)
        if unit is None:
            assert len(pieces) == 1 and pieces[0][2] == -1
        else:
            assert [p[2] for p in pieces] == list(range(unit[0], unit[0] + unit[1]))
    assert not units


def test_few_rows_over_a_long_context_use_the_whole_gpu(lib):
    indptr, last = lay([65536])
    offsets, items, merge, slots = lib.plan_prefill_host(indptr, last, np.array([0, 1], np.int32),
                                                         8, 1, 152)
    assert len(offsets) - 1 > 76 and len(merge) == 1
    # prompts that fill it stay whole
    indptr, last = lay([4096] * 8)
    qo = (4096 * np.arange(9)).astype(np.int32)
    assert lib.plan_prefill_host(indptr, last, qo, 4, 8, 152)[3] == 0


def test_plan_refusals(lib):
    """Each refused on the host, before any CUDA call."""
    arr = lambda v: np.array(v, np.int32)  # noqa: E731

    def plan(indptr=(0, 1), last=(3,), qo=(0, 2), hq=8, hkv=2, d=128, page=16, q=1, kv=1, ws=256,
             indices=256, batch=None):
        a, l, r = arr(indptr), arr(last), arr(qo)
        out = ctypes.c_void_p()
        rc = lib.library().fa_prefill_plan(
            a.ctypes.data, indices, l.ctypes.data, r.ctypes.data, len(a) - 1 if batch is None else batch,
            hq, hkv, d, page, q, kv, ws, 1 << 20, None, ctypes.byref(out))
        assert not out.value
        return rc

    invalid, unsupported = -1, -2
    for kw, rc in [
            (dict(qo=(0, 4)), invalid), (dict(qo=(1, 2)), invalid), (dict(qo=(0, -1)), invalid),
            (dict(indptr=(1, 2)), invalid), (dict(indptr=(0, -1), qo=(0, 0)), invalid),
            (dict(indptr=(0, 0), qo=(0, 1)), invalid), (dict(last=(0,)), invalid),
            (dict(last=(17,)), invalid), (dict(hq=7), invalid), (dict(hkv=0), invalid),
            (dict(ws=None), invalid), (dict(ws=128), invalid), (dict(indices=None), invalid),
            (dict(batch=-1), invalid), (dict(d=96), unsupported), (dict(page=32), unsupported),
            (dict(hq=6), unsupported), (dict(q=0, kv=0), unsupported), (dict(q=1, kv=2), unsupported),
            (dict(q=2, kv=3), unsupported), (dict(q=3, kv=3), unsupported), (dict(q=9), unsupported)]:
        assert plan(**kw) == rc, kw
    L = lib.library()
    assert L.fa_prefill_plan_destroy(None) == 0
    assert L.fa_prefill_run(None, None, None, 1, 0.0, 1.0, 1.0, None, None, None) == -1
    for name in ("head", "token", "block"):
        f = getattr(L, f"fa_prefill_run_{name}_scales")
        assert f(None, None, None, 1, 0.0, None, None, None, None, None) == -1
    assert L.fa_prefill_check(None, None, None) == -1
    with pytest.raises(lib.FaError):
        lib.plan_prefill_host([0, 1], [3], [0, 4], 4, 2, 8)
    with pytest.raises(ValueError):
        lib.plan_prefill_host([0, 1], [3], [0], 4, 2, 8)


@pytest.mark.gpu
def test_run_refusals(lib, cuda):
    b = Batch([5], [40], 8, 2, 128, BF16, E4M3)
    n = Batch([5], [40], 8, 2, 128)
    p, pn = b.plan(lib), n.plan(lib)
    sh, sb = torch.ones(2, device=cuda), torch.ones((b.num_pages, 2), device=cuda)
    wide = torch.empty((40, 8, 256), dtype=BF16, device=cuda)
    odd = torch.empty(n.q.numel() + 8, dtype=BF16, device=cuda)[4:-4].view(n.q.shape)
    for bad in (lambda: p.run(b.q.float(), b.kv), lambda: p.run(b.q[:-1], b.kv),
                lambda: p.run(b.q.cpu(), b.kv), lambda: p.run(b.q, n.kv),
                lambda: p.run(b.q, b.kv[:, :, :8]), lambda: p.run(b.q, b.kv.cpu()),
                lambda: p.run(wide[..., ::2], b.kv), lambda: p.run(odd, b.kv),
                lambda: p.run(b.q[:1].expand(40, -1, -1), b.kv),
                lambda: p.run(b.q, b.kv, k_scale=-1.0), lambda: p.run(b.q, b.kv, v_scale=float("nan")),
                lambda: p.run(b.q, b.kv, out=b.q), lambda: p.run(b.q, b.kv, out=torch.empty_like(b.q)[:9]),
                lambda: p.run(b.q, b.kv, lse=torch.empty(4, device=cuda)),
                lambda: p.run(b.q, b.kv, out=torch.empty(b.q.numel() + 8, dtype=BF16, device=cuda)[8:]),
                lambda: p.run(b.q, b.kv, out=torch.empty(b.q.shape, dtype=BF16)),
                lambda: p.run(b.q, b.kv, out=torch.empty(b.q.shape, device=cuda)),
                lambda: p.run(b.q, b.kv, lse=torch.empty((40, 8), device=cuda).double()),
                lambda: p.run(b.q, b.kv, lse=torch.empty((40, 8))),
                lambda: p.run_head_scales(b.q, b.kv, sb, sb), lambda: p.run_block_scales(b.q, b.kv, sh, sh),
                lambda: p.run_token_scales(b.q, b.kv, sb, sb),
                lambda: p.run_block_scales(b.q, b.kv, sb, sb.double()),
                lambda: p.run_block_scales(b.q, b.kv, sb.cpu(), sb),
                lambda: pn.run(n.q, n.kv, k_scale=0.5),
                lambda: pn.run_head_scales(n.q, n.kv, sh, sh),
                lambda: pn.run_block_scales(n.q, n.kv, sb[:n.num_pages], sb[:n.num_pages]),
                lambda: n.plan(lib, workspace=torch.empty(16, dtype=torch.uint8, device=cuda)),
                lambda: n.plan(lib, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError, lib.FaError)):
            bad()


@pytest.mark.gpu
def test_another_current_device_is_refused(lib, cuda, monkeypatch):
    b = Batch([0], [4], 8, 2, 128)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=cuda)
    other = torch.cuda.current_device() + 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: other)
    for kw in ({}, {"workspace": ws}):
        with pytest.raises(ValueError):
            b.plan(lib, **kw)

"""Eviction by accumulated weight (plan_evict): the cache, the weights and the scales
afterwards, bit for bit, against the definition; the batch's new layout; and the
steps of a serving program together."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_prefill import BF16, E4M3, F16, Batch

F32 = torch.float32


class Cache:
    def __init__(self, lengths, hkv, d, dtype, seed=0, token_scales=False, weights="random"):
        rng = np.random.default_rng(seed)
        self.lengths = np.asarray(lengths, np.int64)
        self.hkv, self.d, self.dtype = hkv, d, dtype
        pages = (self.lengths + 15) // 16
        self.indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.last = np.where(pages > 0, self.lengths - (pages - 1) * 16, 16).astype(np.int32)
        self.num_pages = int(self.indptr[-1]) + 3
        self.ids = rng.permutation(self.num_pages)[:self.indptr[-1]].astype(np.int32)
        self.indices = torch.from_numpy(self.ids).cuda()
        es = torch.empty(0, dtype=dtype).element_size()
        raw = rng.integers(0, 256, (self.num_pages, 2, 16, hkv, d * es)).astype(np.uint8)
        self.kv = torch.from_numpy(raw).cuda().view(dtype)
        shape = (self.num_pages, hkv, 16)
        w = rng.random(shape).astype(np.float32) ** 8
        if weights == "ties":
            w = np.floor(w * 8) / 8
        elif weights == "odd":  # every kind of float
            w = rng.integers(0, 2 ** 32, shape, dtype=np.uint32).view(np.float32)
            w.flat[::7] = np.float32(-0.0)
            w.flat[::11] = 0.0
            w.flat[::13] = np.inf
        elif weights == "zeros":
            w[:] = 0
        self.w = torch.from_numpy(w.copy()).cuda()
        self.ks = self.vs = None
        if token_scales:
            self.ks, self.vs = (torch.from_numpy(rng.random(shape).astype(np.float32)).cuda()
                                for _ in range(2))

    def plan(self, fa, keep, recent=0, **kw):
        return fa.plan_evict(self.indptr, self.indices, self.last, keep, self.hkv, self.d, 16,
                             recent=recent, kv_data_type=self.dtype, **kw)

    def run(self, p, **kw):
        p.run(self.kv, self.w, k_scales=self.ks, v_scales=self.vs, **kw)

    def state(self):
        t = [self.kv.view(torch.uint8), self.w.view(torch.uint8)]
        if self.ks is not None:
            t += [self.ks.view(torch.uint8), self.vs.view(torch.uint8)]
        return [x.cpu().numpy().copy() for x in t]

    def expected(self, keep, recent):
        """state() after the eviction."""
        s = self.state()
        w = s[1].view(np.float32)
        keep = np.broadcast_to(keep, len(self.lengths))
        recent = np.broadcast_to(recent, len(self.lengths))
        for i, L in enumerate(self.lengths):
            n = min(L, keep[i])
            if n == L:
                continue
            r = min(recent[i], n)
            t = np.arange(L)
            page, slot = self.ids[self.indptr[i] + t // 16], t % 16
            for h in range(self.hkv):
                key = w[page, h, slot][:L - r]
                nan = np.isnan(key)
                key = np.where(nan, np.float32(np.inf), key)
                order = np.lexsort((t[:L - r], -key, ~nan))  # NaN first, then the largest
                kept = np.sort(np.concatenate([order[:n - r], t[L - r:]]))
                for x in s:
                    if x is s[0]:
                        rows = x[page[kept], :, slot[kept], h].copy()
                        x[page[:n], :, slot[:n], h] = rows
                    else:
                        v = x.reshape(*x.shape[:2], 16, 4)
                        rows = v[page[kept], h, slot[kept]].copy()
                        if x is s[1]:
                            v[page, h, slot] = 0
                        v[page[:n], h, slot[:n]] = rows
        return s

    def check(self, fa, keep, recent=0):
        want = self.expected(keep, recent)
        p = self.plan(fa, keep, recent)
        self.run(p)
        assert p.check() == 0
        for got, x in zip(self.state(), want):
            assert np.array_equal(got, x), np.argwhere(got != x)[:4]
        return p


LENGTHS = [100, 0, 16, 17, 15, 1, 300, 33, 64, 1500]


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["random", "ties", "odd", "zeros"])
@pytest.mark.parametrize("keep,recent", [(0, 0), (1, 0), (1, 1), (16, 3), (33, 40), (64, 0),
                                         (200, 16), (5000, 7)])
def test_small(lib, cuda, keep, recent, weights):
    Cache(LENGTHS, 3, 64, BF16, seed=keep, weights=weights).check(lib, keep, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,scales", [(BF16, 128, False), (F16, 64, False), (F32, 128, False),
                                            (F32, 64, False), (E4M3, 64, False), (E4M3, 128, True)])
def test_types(lib, cuda, dtype, d, scales):
    Cache([1000, 40, 700], 4, d, dtype, seed=2, token_scales=scales).check(lib, [130, 64, 699], [9, 0, 64])


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hkv,keep,recent,weights", [
    ([20000], 1, 3000, 100, "random"),       # one cluster of eight CTAs
    ([9000], 2, 8999, 0, "random"),          # nearly all stay
    ([5000, 4100], 8, 700, 700, "ties"),     # the last tokens alone
    ([70000], 1, 2000, 1, "ties"),
    ([130000], 1, 100000, 5, "random"),      # keys beyond a CTA's shared memory
    ([3000] * 40, 8, 1000, 64, "zeros"),     # a CTA each
    ([12000] + [40] * 79, 8, 30, 3, "ties")])  # a CTA each, keys beyond its shared memory
def test_long(lib, cuda, lengths, hkv, keep, recent, weights):
    Cache(lengths, hkv, 64, BF16, seed=3, weights=weights).check(lib, keep, recent)


@pytest.mark.gpu
def test_the_batch_afterwards(lib, cuda):
    c = Cache([100, 0, 16, 17, 300, 5], 2, 64, BF16)
    keep = [40, 3, 16, 16, 1000, 0]
    p = c.plan(lib, keep)
    lengths = [min(a, b) for a, b in zip(c.lengths, keep)]
    assert p.indptr.tolist() == np.concatenate([[0], np.cumsum([-(-n // 16) for n in lengths])]).tolist()
    assert p.last_page_len.tolist() == [n - (-(-n // 16) - 1) * 16 if n else 16 for n in lengths]
    kept = [c.ids[c.indptr[i]:c.indptr[i] + -(-n // 16)] for i, n in enumerate(lengths)]
    assert p.indices.tolist() == np.concatenate(kept).tolist() and p.indices.dtype == torch.int32
    assert sorted(p.freed.tolist() + p.indices.tolist()) == sorted(c.ids.tolist())
    lib.plan(p.indptr, p.indices, p.last_page_len, 2, 2, 64, 16)


@pytest.mark.gpu
def test_stream_and_graph(lib, cuda):
    c = Cache([900, 50], 4, 128, BF16, seed=4)
    want = c.expected(200, 8)
    kv, w = c.kv.clone(), c.w.clone()
    p = c.plan(lib, 200, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c.run(p, stream=side)
    side.synchronize()
    assert all(np.array_equal(a, b) for a, b in zip(c.state(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(p)
    c.kv.copy_(kv)
    c.w.copy_(w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(a, b) for a, b in zip(c.state(), want))


@pytest.mark.gpu
def test_bad_page_ids(lib, cuda):
    """Tokens on them are not moved, nothing outside the request changes, and the
    other heads' and requests' results stay what they are."""
    c = Cache([100, 200], 2, 64, BF16, seed=5)
    other = c.expected(50, 0)
    before = c.state()
    ids = c.indices.clone()
    ids[2] = c.num_pages
    c.indices = ids
    p = c.plan(lib, 50)
    c.run(p)
    assert p.check() == 1 and p.check() == 0
    mine = c.ids[c.indptr[1]:c.indptr[2]]
    now = c.state()
    for a, b in zip(now, other):
        assert np.array_equal(a[mine], b[mine])
    outside = np.setdiff1d(np.arange(c.num_pages), c.ids)
    outside = np.append(outside, c.ids[2])
    for a, b in zip(now, before):
        assert np.array_equal(a[outside], b[outside])


@pytest.mark.gpu
def test_nothing_to_evict(lib, cuda):
    for lengths, keep in (([], 4), ([0, 0], 0), ([5, 16], 16)):
        c = Cache(lengths, 2, 64, BF16)
        c.check(lib, keep)


# ---------------------------------------------------------------- together

@pytest.mark.gpu
@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_a_request_within_a_budget(lib, cuda, kv_dtype):
    """Prompts with images are appended and attended, their weights accumulated, the
    cache trimmed, and a token appended and decoded on what is left: every stage
    against the definition on the stage's own inputs."""
    hq, hkv, d, budget, recent = 8, 2, 128, 96, 16
    b = Batch([0, 0], [150, 260], hq, hkv, d, BF16, kv_dtype, seed=21, extra=8)
    rng = np.random.default_rng(0)
    qkv = torch.from_numpy(rng.standard_normal((b.T, hq + 2 * hkv, d)).astype(np.float32)).cuda().to(BF16)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    rotary = lib.RotaryTable(d, axes=np.repeat([0, 1, 2], [16, 24, 24]))
    pos = torch.from_numpy(rng.integers(0, 300, (3, b.T)).astype(np.int32)).cuda()
    types = dict(q_data_type=BF16, kv_data_type=kv_dtype)
    ks = torch.zeros((b.num_pages, hkv, 16), device=cuda)
    vs = torch.zeros_like(ks)
    scaled = kv_dtype == E4M3

    ap = lib.plan_append(b.indptr, b.indices, b.last, b.qo, hq, hkv, d, 16, rotary=rotary,
                         positions=pos, **types)
    pf = b.plan(lib)
    wp = lib.plan_weights(b.indptr, b.indices, b.last, b.qo, hq, hkv, d, 16, **types)
    ev = lib.plan_evict(b.indptr, b.indices, b.last, budget, hkv, d, 16, recent=recent,
                        kv_data_type=kv_dtype)
    w = torch.zeros((b.num_pages, hkv, 16), device=cuda)
    if scaled:
        qr = ap.run_token_scales(k, v, b.kv, ks, vs, q=q)
        o, lse = pf.run_token_scales(qr, b.kv, ks, vs)
        wp.run_token_scales(qr, b.kv, lse, w, ks)
    else:
        qr = ap.run(k, v, b.kv, q=q)
        o, lse = pf.run(qr, b.kv)
        wp.run(qr, b.kv, lse, w)
    b.q = qr
    of = (lambda half, page, slot: (ks, vs)[half].double()[page, :, slot]) if scaled else None
    b.check(o, lse, of, inexact=scaled)
    # every row's weights sum to one a head, to the logits' errors in fp32: 128 2^-23 of
    # a few units, under 1e-4
    total = w.sum((0, 2))
    assert ((total / (b.T * hq / hkv) - 1).abs() < 1e-4).all()

    c = Cache.__new__(Cache)
    c.__dict__.update(lengths=b.total, hkv=hkv, d=d, dtype=kv_dtype, indptr=b.indptr, last=b.last,
                      ids=b.ids, indices=b.indices, num_pages=b.num_pages, kv=b.kv, w=w,
                      ks=ks if scaled else None, vs=vs if scaled else None)
    want = c.expected(budget, recent)
    c.run(ev)
    assert all(np.array_equal(x, y) for x, y in zip(c.state(), want))

    # one more token a request, in a freed page of its own list's or a new slot
    B = 2
    length = np.minimum(b.total, budget) + 1
    pages = -(-length // 16)
    ids = np.concatenate([b.ids[b.indptr[i]:b.indptr[i] + pages[i]] for i in range(B)])
    n = Batch.__new__(Batch)
    n.__dict__.update(b.__dict__)
    n.indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    n.last = (length - (pages - 1) * 16).astype(np.int32)
    n.ids, n.indices = ids, torch.from_numpy(ids).cuda()
    n.total, n.new, n.ctx, n.T = length, np.array([1, 1]), length - 1, 2
    n.qo = np.array([0, 1, 2], np.int32)
    qkv = torch.from_numpy(rng.standard_normal((2, hq + 2 * hkv, d)).astype(np.float32)).cuda().to(BF16)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    pos = torch.tensor([[150, 260]] * 3, dtype=torch.int32, device=cuda)
    ap = lib.plan_append(n.indptr, n.indices, n.last, n.qo, hq, hkv, d, 16, rotary=rotary,
                         positions=pos, **types)
    dec = lib.plan(n.indptr, n.indices, n.last, hq, hkv, d, 16, **types)
    if scaled:
        n.q = ap.run_token_scales(k, v, n.kv, ks, vs, q=q)
        o, lse = dec.run_token_scales(n.q, n.kv, ks, vs)
    else:
        n.q = ap.run(k, v, n.kv, q=q)
        o, lse = dec.run(n.q, n.kv)
    n.check(o, None, of, inexact=True)  # the decode kernel rounds weights and their sum


@pytest.mark.gpu
def test_cache_beyond_32_bits(lib, cuda):
    """Prefill, weights and eviction over pages behind 2^31 elements: bit for bit what
    they give in a small cache."""
    b = Batch([300], [70], 8, 8, 128, seed=31, garbage=0.0)
    few = torch.tensor([0, 1], dtype=torch.int32)
    pages = 70_000
    big = torch.empty((pages, 2, 16, 8, 128), dtype=BF16, device=cuda)
    assert big.numel() > 2 ** 31
    high = pages - 1 - torch.arange(len(b.ids), dtype=torch.int32, device=cuda)
    big[high.long()] = b.kv[b.indices.long()]
    w = [torch.rand((n, 8, 16), device=cuda) for n in (b.num_pages, pages)]
    w[1][high.long()] = w[0][b.indices.long()]
    out = []
    for kv, ids, wt in ((b.kv.clone(), b.indices, w[0]), (big, high, w[1])):
        o, lse = lib.plan_prefill(b.indptr, ids, b.last, b.qo, 8, 8, 128, 16).run(b.q, kv)
        for rows in (b.qo, few):  # the tcgen05 kernel, and the one of few columns
            n = int(rows[-1])
            lib.plan_weights(b.indptr, ids, b.last, rows, 8, 8, 128, 16).run(
                b.q[b.T - n:].contiguous(), kv, lse[b.T - n:].contiguous(), wt)
        lib.plan_evict(b.indptr, ids, b.last, 100, 8, 128, 16, recent=9).run(kv, wt)
        out.append((o, lse, kv[ids.long()], wt[ids.long()]))
    for x, y in zip(*out):
        assert torch.equal(x, y)


# ---------------------------------------------------------------- refusals

def test_plan_refusals(lib):
    """Each refused on the host, before any CUDA call."""
    arr = lambda v: np.array(v, np.int32)  # noqa: E731

    def plan_rc(indptr=(0, 1), last=(9,), keep=(4,), recent=(2,), hkv=2, d=128, page=16, kv=1,
                ws=256, ws_bytes=1 << 20, indices=256, batch=None):
        a, l, k = arr(indptr), arr(last), arr(keep)
        r = None if recent is None else arr(recent)
        out = ctypes.c_void_p()
        rc = lib.library().fa_evict_plan(
            a.ctypes.data, indices, l.ctypes.data, k.ctypes.data, None if r is None else r.ctypes.data,
            len(a) - 1 if batch is None else batch, hkv, d, page, kv, ws, ws_bytes, None,
            ctypes.byref(out))
        assert not out.value
        return rc

    invalid, unsupported, small = -1, -2, -3
    for kw, rc in [(dict(keep=(-1,)), invalid), (dict(recent=(-1,)), invalid),
                   (dict(indptr=(1, 2)), invalid), (dict(indptr=(0, -1)), invalid),
                   (dict(last=(0,)), invalid), (dict(last=(17,)), invalid), (dict(hkv=0), invalid),
                   (dict(ws=None), invalid), (dict(ws=128), invalid), (dict(indices=None), invalid),
                   (dict(batch=-1), invalid), (dict(d=96), unsupported), (dict(page=32), unsupported),
                   (dict(kv=9), unsupported), (dict(ws_bytes=256), small)]:
        assert plan_rc(**kw) == rc, kw
    L = lib.library()
    assert L.fa_evict_plan_destroy(None) == 0
    assert L.fa_evict_run(None, None, 1, None, None, None, None) == -1
    assert L.fa_evict_check(None, None, None) == -1
    assert L.fa_evict_workspace_size(4, 1000, 8) >= 4 * 1000 * 8
    for bad in ((-1, 5, 1), (1, -5, 1), (1, 5, 0)):
        assert L.fa_evict_workspace_size(*bad) == 0


@pytest.mark.gpu
def test_run_refusals(lib, cuda):
    c = Cache([100], 2, 64, E4M3, token_scales=True)
    n = Cache([100], 2, 64, BF16)
    p, pn = c.plan(lib, 9), n.plan(lib, 9)
    before = c.state()
    block = torch.ones((c.num_pages, 2), device=cuda)
    for bad in (lambda: p.run(n.kv, c.w), lambda: p.run(c.kv[:, :, :8], c.w), lambda: p.run(c.kv.cpu(), c.w),
                lambda: p.run(c.kv, c.w[:-1]), lambda: p.run(c.kv, c.w.double()),
                lambda: p.run(c.kv, c.w.cpu()), lambda: p.run(c.kv, c.w, k_scales=c.ks),
                lambda: p.run(c.kv, c.w, k_scales=block, v_scales=block),
                lambda: pn.run(n.kv, n.w, k_scales=n.w.clone(), v_scales=n.w.clone()),
                lambda: c.plan(lib, -1), lambda: c.plan(lib, [1, 2]), lambda: c.plan(lib, 4, recent=-1),
                lambda: c.plan(lib, 4, workspace=torch.empty(16, dtype=torch.uint8, device=cuda)),
                lambda: c.plan(lib, 4, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError, lib.FaError)):
            bad()
    torch.cuda.synchronize()
    assert all(np.array_equal(a, b) for a, b in zip(c.state(), before))

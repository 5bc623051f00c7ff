"""Attention weights accumulated per cached token (plan_weights) against the
definition in 64 bits, and their refusals.

Tolerance.  A weight is exp(s - lse) of a logit in fp32: the logit's error as in
test_prefill.py, D 2^-23 times the sum of its products' magnitudes and 2^-21 of it;
the given lse is a float and is multiplied by log2 e (2^-23 of it); the exponential
2^-22.  Those relative errors hold for a sum of weights too, plus 2^-24 for each of its
additions (columns / 8 in a lane, 3 across lanes, one to memory) and the rounding
of the stored sum.
"""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_prefill import BF16, E4M3, F16, LENGTHS, Batch


def plan(b, lib, **kw):
    return lib.plan_weights(b.indptr, b.indices, b.last, b.qo, b.hq, b.hkv, b.d, 16,
                            q_data_type=b.q_dtype, kv_data_type=b.kv_dtype, **kw)


def logits(b, i, scale_of, sm):
    """Request i's logits [hq, rows, tokens] masked, the sums of magnitudes, and its
    tokens' pages and slots."""
    n, L, G = int(b.new[i]), int(b.total[i]), b.hq // b.hkv
    t = torch.arange(L, device="cuda")
    page = b.indices[b.indptr[i]:b.indptr[i + 1]].long()[t // 16]
    k = b.kv.double()[page, 0, t % 16]
    if scale_of is not None:
        k = k * scale_of(page, t % 16)[..., None]
    q = b.q[b.qo[i]:b.qo[i + 1]].double().transpose(0, 1)
    kh = k.transpose(0, 1).repeat_interleave(G, 0)
    seen = t[None, :] <= L - n + torch.arange(n, device="cuda")[:, None]
    s = (q @ kh.transpose(1, 2) * sm).masked_fill(~seen, -float("inf"))
    size = (q.abs() @ kh.abs().transpose(1, 2) * sm).masked_fill(~seen, 0)
    return s, size, page, t % 16


def exact_lse(b, scale_of=None, sm=None):
    sm = b.d ** -0.5 if sm is None else sm
    out = torch.full((b.T, b.hq), -float("inf"), dtype=torch.float64, device="cuda")
    for i in range(len(b.total)):
        if b.new[i] and b.total[i]:
            out[b.qo[i]:b.qo[i + 1]] = logits(b, i, scale_of, sm)[0].logsumexp(-1).T
    return out.float()


def check(b, got, before, lse, scale_of=None, sm=None):
    sm = b.d ** -0.5 if sm is None else sm
    want, bound = before.double(), torch.zeros_like(before, dtype=torch.float64)
    for i in range(len(b.total)):
        if not (b.new[i] and b.total[i]):
            continue
        s, size, page, slot = logits(b, i, scale_of, sm)
        l = lse[b.qo[i]:b.qo[i + 1]].T.double()[..., None]
        l = torch.where(l == -float("inf"), -l, l)
        w = (s - l).exp()
        err = size * (b.d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -22 * l.abs().nan_to_num(0, 0) + 2.0 ** -21
        G = b.hq // b.hkv
        per = w.view(b.hkv, G, *w.shape[1:]).sum((1, 2))
        slack = (w * err).nan_to_num(0).view(b.hkv, G, *w.shape[1:]).sum((1, 2))
        adds = w.shape[1] * G / 8 + 5
        want[page, :, slot] += per.T
        bound[page, :, slot] += (slack + adds * 2.0 ** -24 * per).T
    bound += 2.0 ** -24 * (want.abs() + before.abs()) + 2.0 ** -120
    bad = ~((got.double() - want).abs() <= bound * 1.001)
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], want[bad][:4], bound[bad][:4])
    untouched = bound <= 2.0 ** -24 * (want.abs() + before.abs()) + 2.0 ** -120
    assert torch.equal(got[untouched], before[untouched])


def fresh(b):
    g = torch.Generator(device="cuda").manual_seed(3)
    return torch.rand((b.num_pages, b.hkv, 16), generator=g, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("dtype,d,hq,hkv", [
    (BF16, 128, 32, 8), (BF16, 128, 8, 1), (F16, 128, 3, 3), (F16, 64, 10, 5), (BF16, 64, 8, 2),
    (BF16, 64, 1, 1)])
def test_native(lib, cuda, dtype, d, hq, hkv, lengths):
    b = Batch(*LENGTHS[lengths], hq, hkv, d, dtype, seed=lengths)
    lse = exact_lse(b)
    w = fresh(b)
    before = w.clone()
    p = plan(b, lib)
    assert p.run(b.q, b.kv, lse, w) is w
    assert p.check() == 0
    check(b, w, before, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 128), (BF16, 64), (F16, 64)])
@pytest.mark.parametrize("mode", ["tensor", "head", "token", "block"])
def test_e4m3(lib, cuda, mode, dtype, d):
    b = Batch([0, 40, 300, 1000], [70, 1, 130, 1], 16, 4, d, dtype, E4M3, seed=7)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda") * 0.2 + 0.001  # noqa: E731
    s = {"head": rand(4), "token": rand(b.num_pages, 4, 16), "block": rand(b.num_pages, 4),
         "tensor": torch.tensor([0.11], device=cuda)}[mode]
    of = {"head": lambda page, slot: s.double().expand(len(page), 4),
          "tensor": lambda page, slot: s.double().expand(len(page), 4),
          "token": lambda page, slot: s.double()[page, :, slot],
          "block": lambda page, slot: s.double()[page]}[mode]
    lse = exact_lse(b, of)
    w = fresh(b)
    before, p = w.clone(), plan(b, lib)
    if mode == "tensor":
        p.run(b.q, b.kv, lse, w, k_scale=float(s[0]))
    else:
        getattr(p, f"run_{mode}_scales")(b.q, b.kv, lse, w, s)
    check(b, w, before, lse, of)


@pytest.mark.gpu
def test_weights_of_a_decode_step_sum_to_one(lib, cuda):
    """After plan.run, one row a request (qo_indptr None), an empty request among
    them: each row's weights sum to 1 for every head of a group."""
    b = Batch([99, 0, 4000, 15], [1, 0, 1, 1], 32, 8, 128, seed=4)
    q = torch.randn((4, 32, 128), device=cuda).to(BF16)
    o, lse = lib.plan(b.indptr, b.indices, b.last, 32, 8, 128, 16).run(q, b.kv)
    w = torch.zeros((b.num_pages, 8, 16), device=cuda)
    p = lib.plan_weights(b.indptr, b.indices, b.last, None, 32, 8, 128, 16)
    p.run(q, b.kv, lse, w)
    for i in (0, 2, 3):
        total = w[b.indices[b.indptr[i]:b.indptr[i + 1]].long()].sum((0, 2))
        # lse of the decode kernel: ln of a sum of weights rounded to bf16 (2^-8)
        assert ((total - 4).abs() <= 4 * 2.0 ** -8 * 1.01).all()
    assert torch.isfinite(w).all() and abs(float(w.sum()) - 3 * 32) < 3 * 32 * 2.0 ** -8


@pytest.mark.gpu
def test_rows_before_the_first_token_and_rows_of_minus_infinity(lib, cuda):
    """More rows than tokens: the first see nothing; an lse of -inf adds nothing."""
    b = Batch([0], [5], 4, 2, 64, seed=5)
    q = torch.randn((9, 4, 64), device=cuda).to(BF16)
    q[4:] = b.q
    lse = torch.full((9, 4), -float("inf"), device=cuda)
    lse[4:] = exact_lse(b)
    w = fresh(b)
    before = w.clone()
    p = lib.plan_weights(b.indptr, b.indices, b.last, [0, 9], 4, 2, 64, 16)
    p.run(q, b.kv, lse, w)
    check(b, w, before, lse[4:])
    lse[6] = -float("inf")
    w2 = before.clone()
    p.run(q, b.kv, lse, w2)
    check(b, w2, before, lse[4:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d,ctx,new", [(1, 1, 64, 50, 1), (4, 2, 128, 50, 1), (8, 2, 64, 37, 1),
                                              (8, 2, 128, 100, 5), (4, 4, 64, 300, 33)])
def test_logits_of_minus_infinity_weigh_nothing(lib, cuda, dtype, hq, hkv, d, ctx, new):
    """An infinite element of K against negative elements of q: the token's weights are
    0, whatever number of columns a tile is filled up with."""
    b = Batch([ctx], [new], hq, hkv, d, dtype, seed=31)
    b.q[..., 3] = -1
    page = b.indices.long()[1]
    b.kv[page, 0, 5, :, 3] = float("inf")
    lse, w = exact_lse(b), fresh(b)
    assert torch.isfinite(lse).all()
    before = w.clone()
    plan(b, lib).run(b.q, b.kv, lse, w)
    assert torch.equal(w[page, :, 5], before[page, :, 5])
    check(b, w, before, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1, 1], [70, 2, 130]])
def test_scales_behind_the_last_token_are_ignored(lib, cuda, new):
    b = Batch([0, 40, 300], new, 8, 2, 128, BF16, E4M3, seed=32)
    g = torch.Generator(device="cuda").manual_seed(2)
    s = torch.rand((b.num_pages, 2, 16), generator=g, device="cuda") * 0.1 + 0.001
    s[(b.kv.view(torch.uint8)[:, 0, :, :, 0] == 127).transpose(1, 2)] = float("nan")
    of = lambda page, slot: s.double()[page, :, slot]  # noqa: E731
    lse, w = exact_lse(b, of), fresh(b)
    before = w.clone()
    plan(b, lib).run_token_scales(b.q, b.kv, lse, w, s)
    check(b, w, before, lse, of)


@pytest.mark.gpu
def test_strides_stream_and_graph(lib, cuda):
    b = Batch([0, 500], [30, 20], 16, 4, 128, seed=6)
    lse = exact_lse(b, sm=0.1)
    p = plan(b, lib)
    fused = torch.full((b.T, 24, 128), float("nan"), dtype=BF16, device=cuda)
    fused[:, 3:19] = b.q
    w0 = fresh(b)
    a, c, d = w0.clone(), w0.clone(), w0.clone()
    p.run(b.q, b.kv, lse, a, sm_scale=0.1)
    check(b, a, w0, lse, sm=0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    p.run(fused[:, 3:19], b.kv, lse, c, sm_scale=0.1, stream=side)
    side.synchronize()
    assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(b.q, b.kv, lse, d, sm_scale=0.1)
    d.copy_(w0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    p.run(b.q, b.kv, lse, a, sm_scale=0.1)
    assert torch.equal(a, d)


@pytest.mark.gpu
def test_shared_pages_get_the_weights_of_all(lib, cuda):
    b = Batch([64, 64], [20, 9], 8, 2, 128, seed=14)
    b.ids[b.indptr[1]:b.indptr[1] + 4] = b.ids[:4]
    b.indices = torch.from_numpy(b.ids).cuda()
    lse = exact_lse(b)
    w = fresh(b)
    before = w.clone()
    plan(b, lib).run(b.q, b.kv, lse, w)
    check(b, w, before, lse)


@pytest.mark.gpu
def test_bad_page_ids_are_skipped(lib, cuda):
    b = Batch([0, 200], [40, 150], 8, 2, 128, seed=13)
    lse = exact_lse(b)
    good, bad = fresh(b), fresh(b)
    before = good.clone()
    plan(b, lib).run(b.q, b.kv, lse, good)
    at = int(b.indptr[1]) + 3
    for value in (-1, b.num_pages, 2 ** 31 - 1):
        ids = b.indices.clone()
        ids[at] = value
        bad.copy_(before)
        p = lib.plan_weights(b.indptr, ids, b.last, b.qo, 8, 2, 128, 16)
        p.run(b.q, b.kv, lse, bad)
        assert p.check() == 1 and p.check() == 0
        assert torch.equal(bad[b.ids[at]], before[b.ids[at]])
        bad[b.ids[at]] = good[b.ids[at]]
        assert torch.equal(bad, good)


@pytest.mark.gpu
def test_no_rows(lib, cuda):
    for ctx, new in (([], []), ([5, 0], [0, 0])):
        b = Batch(ctx, new, 8, 2, 64)
        w = fresh(b)
        before = w.clone()
        plan(b, lib).run(b.q, b.kv, torch.empty((0, 8), device=cuda), w)
        assert torch.equal(w, before)


# ---------------------------------------------------------------- refusals

def test_plan_refusals(lib):
    """Each refused on the host, before any CUDA call."""
    arr = lambda v: np.array(v, np.int32)  # noqa: E731

    def plan_rc(indptr=(0, 1), last=(3,), qo=(0, 2), hq=8, hkv=2, d=128, page=16, q=1, kv=1, ws=256,
                indices=256, batch=None):
        a, l, r = arr(indptr), arr(last), arr(qo)
        out = ctypes.c_void_p()
        rc = lib.library().fa_weights_plan(
            a.ctypes.data, indices, l.ctypes.data, r.ctypes.data, len(a) - 1 if batch is None else batch,
            hq, hkv, d, page, q, kv, ws, 1 << 20, None, ctypes.byref(out))
        assert not out.value
        return rc

    invalid, unsupported = -1, -2
    for kw, rc in [
            (dict(qo=(1, 2)), invalid), (dict(qo=(0, -1)), invalid), (dict(indptr=(1, 2)), invalid),
            (dict(indptr=(0, -1)), invalid), (dict(last=(0,)), invalid), (dict(last=(17,)), invalid),
            (dict(hq=7), invalid), (dict(hkv=0), invalid), (dict(ws=None), invalid),
            (dict(ws=128), invalid), (dict(indices=None), invalid), (dict(batch=-1), invalid),
            (dict(d=96), unsupported), (dict(page=32), unsupported), (dict(hq=6), unsupported),
            (dict(q=0, kv=0), unsupported), (dict(q=1, kv=2), unsupported),
            (dict(q=3, kv=3), unsupported), (dict(q=9), unsupported)]:
        assert plan_rc(**kw) == rc, kw
    L = lib.library()
    assert L.fa_weights_plan_destroy(None) == 0
    assert L.fa_weights_run(None, None, None, 1, 0.0, 1.0, None, None, None) == -1
    for name in ("head", "token", "block"):
        f = getattr(L, f"fa_weights_run_{name}_scales")
        assert f(None, None, None, 1, 0.0, None, None, None, None) == -1
    assert L.fa_weights_check(None, None, None) == -1
    assert L.fa_weights_workspace_size(4, 1000) > 0
    assert L.fa_weights_workspace_size(-1, 1000) == 0 == L.fa_weights_workspace_size(1, -1)


@pytest.mark.gpu
def test_run_refusals(lib, cuda):
    b = Batch([5], [40], 8, 2, 128, BF16, E4M3)
    n = Batch([5], [40], 8, 2, 128)
    p, pn = plan(b, lib), plan(n, lib)
    lse, w = torch.zeros((40, 8), device=cuda), fresh(b)
    before = w.clone()
    sh, sb = torch.ones(2, device=cuda), torch.ones((b.num_pages, 2), device=cuda)
    for bad in (lambda: p.run(b.q.float(), b.kv, lse, w), lambda: p.run(b.q[:-1], b.kv, lse, w),
                lambda: p.run(b.q.cpu(), b.kv, lse, w), lambda: p.run(b.q, n.kv, lse, w),
                lambda: p.run(b.q, b.kv[:, :, :8], lse, w), lambda: p.run(b.q, b.kv.cpu(), lse, w),
                lambda: p.run(b.q, b.kv, lse[:-1], w), lambda: p.run(b.q, b.kv, lse.double(), w),
                lambda: p.run(b.q, b.kv, lse.cpu(), w), lambda: p.run(b.q, b.kv, lse, w[:-1]),
                lambda: p.run(b.q, b.kv, lse, w.double()), lambda: p.run(b.q, b.kv, lse, w.cpu()),
                lambda: p.run(b.q, b.kv, lse, w.transpose(1, 2)),
                lambda: p.run(b.q, b.kv, lse, w, k_scale=float("nan")),
                lambda: p.run_head_scales(b.q, b.kv, lse, w, sb),
                lambda: p.run_block_scales(b.q, b.kv, lse, w, sh),
                lambda: p.run_token_scales(b.q, b.kv, lse, w, sb),
                lambda: pn.run(n.q, n.kv, lse, w, k_scale=0.5),
                lambda: pn.run_head_scales(n.q, n.kv, lse, w, sh),
                lambda: plan(n, lib, workspace=torch.empty(16, dtype=torch.uint8, device=cuda)),
                lambda: plan(n, lib, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError, lib.FaError)):
            bad()
    torch.cuda.synchronize()
    assert torch.equal(w, before)

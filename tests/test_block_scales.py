"""Decode over an E4M3 cache with one scale per block (page, kv head) against
the float64 oracle on the dequantised cache, on every plan kind.

Tolerance of an output element, for weights w over tokens with values v:
half a step of the output's type (bf16 2^-8, f16 2^-11) of itself; 3 * 2^-11 of
sum w |v| for the f16 rounding of a weight, of a weight times its block's
scale, and of the weights' sum; twice the logit error, 2e-4, of sum w |v|; and
2^-25 of the largest |v| for each token whose weight is below f16's normal range
(half its smallest step), of at most as many as the request has.  lse: the
weights' rounding 2^-11, the logit error 1e-4, fp32's rounding of the value.
"""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_decode_fa_gb300 import workloads as W
from tests.helpers import as_bits

E4M3 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(lengths, counts, hq, hkv, d, q_dtype, seed, device, spread=2.0, pow2=True, zero=0.05):
    """A batch whose blocks' scales are spread over 2^+-spread, some of V's
    and (rarely) K's 0; NaN codes in every slot past a request's end."""
    if counts is None:
        b = W.make_batch(batch_lengths=lengths, num_qo_heads=hq, num_kv_heads=hkv, head_dim=d,
                         q_dtype=q_dtype, kv_dtype=E4M3, seed=seed, device=device)
    else:
        b = W.make_ragged_q_batch(batch_lengths=lengths, q_counts=counts, num_qo_heads=hq,
                                  num_kv_heads=hkv, head_dim=d, q_dtype=q_dtype, kv_dtype=E4M3,
                                  seed=seed, device=device)
    rng = np.random.default_rng(seed)
    shape = (b.num_pages, hkv)
    u = rng.uniform(-1, 1, (2,) + shape) * np.array([min(spread, 1.5), spread])[:, None, None]
    s = 2.0 ** (-6.5 + (np.rint(u) if pow2 else u))
    if pow2:
        s *= 2.0 ** 0.5
    s[1][rng.random(shape) < zero] = 0
    s[0][rng.random(shape) < zero / 5] = 0
    b.extra["ks"], b.extra["vs"] = (torch.from_numpy(x.astype(np.float32)).to(device) for x in s)
    raw = b.paged_kv.view(torch.uint8)
    ids = b.indices.cpu().numpy()
    for i, n in enumerate(b.lengths):
        if n % 16:
            raw[int(ids[b.indptr[i + 1] - 1]), :, int(n % 16):] = 0x7f
    return b


def plan(lib, b):
    args = (b.num_qo_heads, b.num_kv_heads, b.head_dim, 16)
    kw = dict(q_data_type=b.q.dtype, kv_data_type=E4M3)
    if "qo_indptr" in b.extra:
        return lib.plan_ragged_q(b.indptr, b.indices, b.last_page_len, b.extra["qo_indptr"], *args,
                                 **kw)
    return lib.plan(b.indptr, b.indices, b.last_page_len, *args, **kw)


def reference(b):
    """(o, lse, sum w |v|, per-row largest |v| times 2^-25 tokens)."""
    kv = b.paged_kv.float()
    kv *= torch.stack([b.extra["ks"], b.extra["vs"]], 1)[:, :, None, :, None]
    qb, qc = as_bits(b.q)
    ids, indptr = b.indices.cpu().numpy(), b.indptr.numpy()
    qo = b.extra.get("qo_indptr", np.arange(b.batch + 1))

    def run(x):
        return oracle.batch_decode_ragged_q(qb, qc, x.cpu().numpy(), oracle.F32, indptr, ids,
                                            b.last_page_len.numpy(), qo, b.num_qo_heads,
                                            b.num_kv_heads, b.head_dim, 16)

    # the plain oracle for a request without a context, which has a row
    def plain(x):
        return oracle.batch_decode(qb, qc, x.cpu().numpy(), oracle.F32, indptr, ids,
                                   b.last_page_len.numpy(), b.num_qo_heads, b.num_kv_heads,
                                   b.head_dim, 16)

    fn = run if "qo_indptr" in b.extra else plain
    o, lse = fn(kv)
    mag = kv.clone()
    mag[:, 1].abs_()
    a, _ = fn(mag)
    big = kv[:, 1].nan_to_num().abs().amax((1, 3)).double().cpu().numpy()  # [pages, hkv]
    tail = np.zeros(lse.shape)
    g = b.num_qo_heads // b.num_kv_heads
    for i in range(b.batch):
        pages = ids[indptr[i]:indptr[i + 1]]
        if len(pages):
            tail[qo[i]:qo[i + 1]] = np.repeat(big[pages].max(0), g) * int(b.lengths[i]) * 2.0 ** -25
    return o, lse, a, tail


def check(b, o, lse, ref):
    ro, rl, a, tail = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    o, lse = o.reshape(ro.shape), lse.reshape(rl.shape)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty)
    tol = HALF[b.q.dtype] * np.abs(ro) + (3 * 2.0 ** -11 + 2e-4) * a * 1.01 + tail[..., None]
    if b.q.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # f16's subnormal outputs
    bad = ~(np.abs(o - ro) <= tol + 1e-30)
    assert not bad.any(), (np.argwhere(bad)[:4], o[bad][:4], ro[bad][:4], tol[bad][:4])
    tol = 2.0 ** -11 + 1e-4 + 2.0 ** -23 * np.abs(rl[~empty])
    assert (np.abs(lse[~empty] - rl[~empty]) <= tol).all(), np.abs(lse[~empty] - rl[~empty]).max()


def run(p, b, **kw):
    o, lse = p.run_block_scales(b.q, b.paged_kv, b.extra["ks"], b.extra["vs"], **kw)
    torch.cuda.synchronize()
    return o, lse


LENGTHS = [1, 0, 16, 17, 250, 1000, 33, 611, 3000]

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spread,pow2", [(0.0, True), (3.0, True), (14.0, True), (3.0, False)])
@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_against_oracle(lib, cuda, group, head_dim, q_dtype, spread, pow2):
    if q_dtype == torch.float16 and spread > 8:
        spread = 8.0  # f16 outputs end at 65504
    b = make(LENGTHS, None, 3 * group, 3, head_dim, q_dtype, 11 * group + head_dim, cuda, spread,
             pow2)
    p = plan(lib, b)
    o, lse = run(p, b)
    assert p.check() == 0 and p.info["num_merge_units"] > 0
    check(b, o, lse, reference(b))
    o2, lse2 = run(p, b)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("merge", ["fused", "kernel"])
@pytest.mark.parametrize("buckets", ["default", "all"])
@pytest.mark.parametrize("group,counts", [(8, [1, 4, 2, 0, 3, 4, 1, 1, 2]),
                                          (4, [2, 8, 1, 0, 3, 6, 2, 1, 5]),
                                          (2, [4, 12, 2, 0, 5, 16, 4, 1, 9]),
                                          (1, [8, 20, 4, 0, 9, 32, 8, 1, 17]),
                                          (1, [8, 1, 0, 3, 8, 5, 2, 7, 4]),
                                          (2, [4, 1, 0, 3, 2, 4, 2, 1, 4]),
                                          (4, [2, 1, 0, 1, 2, 2, 2, 1, 2]),
                                          (8, [1, 1, 0, 1, 1, 1, 1, 0, 1])])
def test_ragged_q(lib, cuda, monkeypatch, group, counts, buckets, merge):
    """Every ragged kernel: one tile, the column splits of two, three and four
    warps, in one launch or a bucket each."""
    if buckets == "all":
        monkeypatch.setenv("FADECODE_BUCKETS", "all")
    else:
        monkeypatch.delenv("FADECODE_BUCKETS", raising=False)
    if merge == "kernel":
        monkeypatch.setenv("FADECODE_MERGE", "kernel")
    else:
        monkeypatch.delenv("FADECODE_MERGE", raising=False)
    lengths = [3000, 40, 2500, 17, 1000, 611, 5000, 9, 250]
    b = make(lengths, counts, 2 * group, 2, 128, torch.bfloat16, 7 + group, cuda, spread=5.0)
    p = plan(lib, b)
    o, lse = run(p, b)
    assert p.check() == 0
    check(b, o, lse, reference(b))


@pytest.mark.parametrize("group,q_len", [(1, 2), (1, 4), (1, 8), (2, 2), (2, 4), (4, 2), (8, 3)])
def test_multi_token(lib, cuda, group, q_len):
    lengths = [8, 16, 17, 250, 1000, 33, 2000]
    b = make(lengths, [q_len] * len(lengths), 2 * group, 2, 128, torch.bfloat16, 31 + group, cuda)
    p = lib.plan_multi_token(b.indptr, b.indices, b.last_page_len, q_len, 2 * group, 2, 128, 16,
                             q_data_type=torch.bfloat16, kv_data_type=E4M3)
    q = b.q.view(len(lengths), q_len, 2 * group, 128)
    o, lse = p.run_block_scales(q, b.paged_kv, b.extra["ks"], b.extra["vs"])
    torch.cuda.synchronize()
    assert o.shape == q.shape and lse.shape == q.shape[:-1] and p.check() == 0
    check(b, o, lse, reference(b))


@pytest.mark.parametrize("group", [2, 4, 8])
def test_equal_scales_are_a_per_tensor_scale(lib, cuda, group):
    """One power of two for every block, where both runs multiply on the tensor
    cores: the same f16 weights, but summed here before they are rounded, by
    the per-tensor kernel after - 2^-11 of the sum at most, in lse and in o, and
    the two outputs' own rounding."""
    b = make(LENGTHS, None, 2 * group, 2, 128, torch.bfloat16, 3, cuda)
    b.extra["ks"].fill_(2.0 ** -5)
    b.extra["vs"].fill_(2.0 ** -3)
    p = plan(lib, b)
    assert p.info["tensor_cores"] == 1
    o, lse = run(p, b)
    ref_o, ref_lse = p.run(b.q, b.paged_kv, k_scale=2.0 ** -5, v_scale=2.0 ** -3)
    torch.cuda.synchronize()
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), empty)
    assert ((lse - ref_lse)[~empty].abs() <= 2.0 ** -11 + 2.0 ** -22 * ref_lse[~empty].abs()).all()
    o, ref_o = o.float(), ref_o.float()
    assert ((o - ref_o).abs() <= (2 * 2.0 ** -8 + 2.0 ** -10) * ref_o.abs() + 1e-30).all()


@pytest.mark.parametrize("tiny,first", [(30, True), (30, False), (60, True), (60, False)])
@pytest.mark.parametrize("group,head_dim,counts", [(2, 128, None), (8, 128, None), (1, 128, None),
                                                   (4, 64, None), (8, 128, [4, 3])])
def test_attended_blocks_of_small_scale(lib, cuda, group, head_dim, counts, tiny, first):
    """Blocks the softmax ignores (a logit lower by 300: weight 0) have V
    scales 2^tiny above those it attends to, before or after them: the
    attended values keep their precision all the same."""
    lengths = [300, 700]
    b = make(lengths, counts, 2 * group, 2, head_dim, torch.bfloat16, 5, cuda, zero=0.0)
    b.q.abs_().clamp_(0.5, 2.0)
    raw = b.paged_kv.view(torch.uint8)
    raw[:, 0] &= 0x7f
    raw[:, 0] = torch.where(raw[:, 0] > 0x40, 0x40, raw[:, 0])  # K codes 0 .. 2
    b.extra["ks"].fill_(2.0 ** -6)
    ids = b.indices.cpu().numpy()
    for i in range(2):
        pages = ids[b.indptr[i]:b.indptr[i + 1]]
        half = len(pages) // 2 if counts is None else len(pages) - 2
        off = pages[:half] if (first or counts is not None) else pages[half:]
        if not first and counts is not None:
            off = pages[1:half]
        off = torch.from_numpy(off.astype(np.int64)).to(cuda)
        kc = raw[off, 0] & 0
        raw[off, 0] = kc + (0x7e | 0x80)         # K code -448
        b.extra["ks"][off] = 4.0
        b.extra["vs"][off] = b.extra["vs"][off] * 2.0 ** tiny
    p = plan(lib, b)
    o, lse = run(p, b)
    ref = reference(b)
    # no token has a weight between 0 and f16's normal range
    check(b, o, lse, (ref[0], ref[1], ref[2], ref[3] * 0))


def test_bad_page_ids_and_empty(lib, cuda):
    b = make([40, 0, 70], None, 8, 2, 128, torch.bfloat16, 24, cuda)
    good = b.indices.clone()
    b.indices[1] = b.num_pages + 5
    b.indices[4] = -7
    p = plan(lib, b)
    run(p, b)
    assert p.check() == 1
    b.indices.copy_(good)
    o, lse = run(p, b)
    assert p.check() == 0
    check(b, o, lse, reference(b))
    e = lib.plan(np.zeros(3, np.int32), b.indices[:0], np.ones(2, np.int32), 8, 2, 128, 16,
                 q_data_type=torch.bfloat16, kv_data_type=E4M3)
    o, lse = e.run_block_scales(b.q[:2], b.paged_kv, b.extra["ks"], b.extra["vs"])
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_graph_capture_and_other_stream(lib, cuda):
    b = make([3000, 17, 0, 900], None, 16, 4, 128, torch.bfloat16, 131, cuda)
    p = plan(lib, b)
    o, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=cuda)
    run(p, b, out=o, lse=lse)
    ref = o.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run_block_scales(b.q, b.paged_kv, b.extra["ks"], b.extra["vs"], out=o, lse=lse)
    for _ in range(3):
        o.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o.zero_()
    p.run_block_scales(b.q, b.paged_kv, b.extra["ks"], b.extra["vs"], out=o, return_lse=False,
                       stream=side)
    side.synchronize()
    assert torch.equal(o, ref[0])


@pytest.mark.parametrize("env", [("FADECODE_POOL", "0.25"), ("FADECODE_PLAN", "stream"),
                                 ("FADECODE_KERNEL", "simt")], ids=lambda e: e[0])
@pytest.mark.parametrize("group,head_dim", [(1, 128), (8, 128), (2, 64), (4, 64), (8, 64)])
def test_other_plans(lib, cuda, monkeypatch, group, head_dim, env):
    """Segments claimed at run time, the stream plan, and a plan whose plain
    kernel is the CUDA-core one."""
    monkeypatch.setenv(*env)
    lengths = [60000, 3, 0, 16, 17, 30000] + list(range(0, 400, 7))
    b = make(lengths, None, 3 * group, 3, head_dim, torch.bfloat16, 17, cuda, spread=4.0)
    p = plan(lib, b)
    if env[0] == "FADECODE_POOL":
        assert p.info["num_pool_segments"] > 0
    o, lse = run(p, b)
    assert p.check() == 0
    check(b, o, lse, reference(b))
    for _ in range(3):
        o2, lse2 = run(p, b)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("batch,group,prefix_pages,spread", [(3, 4, 40, 3.0), (40, 8, 33, 0.0),
                                                             (5, 1, 1, 3.0), (70, 2, 300, 8.0)])
def test_cascade(lib, cuda, batch, group, prefix_pages, spread, q_dtype):
    """A shared prefix and own pages of every length in one block-scaled cache,
    against the oracle over the full page lists."""
    b = W.make_cascade_batch(prefix_pages=prefix_pages,
                             suffix_lengths=[(7 * i) % 61 for i in range(batch)],
                             num_qo_heads=3 * group, num_kv_heads=3, head_dim=128, dtype=q_dtype,
                             kv_dtype=E4M3, seed=batch, device=cuda)
    rng = np.random.default_rng(batch)
    s = 2.0 ** (-6 + np.rint(rng.uniform(-1, 1, (2, b.num_pages, 3))
                             * np.array([min(spread, 1.5), spread])[:, None, None]))
    s[1][rng.random(s[1].shape) < 0.05] = 0
    b.extra["ks"], b.extra["vs"] = (torch.from_numpy(x.astype(np.float32)).to(cuda) for x in s)
    p = lib.cascade_plan(*W.cascade_parts(b), 3 * group, 3, 128, 16, q_data_type=q_dtype,
                         kv_data_type=E4M3)
    ref = reference(b)
    for _ in range(2):
        o, lse = run(p, b)
        assert p.check() == 0
        # the suffix' own output passes through q's type once more
        ro, rl, a, tail = ref
        check(b, o, lse, (ro, rl, a + HALF[q_dtype] / (3 * 2.0 ** -11) * a, tail))
    plain, _ = p.run(b.q, b.paged_kv, k_scale=0.02, v_scale=0.02)   # the other pass still runs
    assert torch.isfinite(plain).all()
    with pytest.raises(ValueError):
        p.run_block_scales(b.q, b.paged_kv, b.extra["ks"][:-1], b.extra["vs"])
    with pytest.raises(ValueError):
        p.run_block_scales(b.q, b.paged_kv[:, :, :8].contiguous(), b.extra["ks"], b.extra["vs"])


@pytest.mark.parametrize("lengths,counts,hq,hkv,d", [
    ([9000, 47000], [5, 6], 8, 2, 128), ([40000], None, 8, 1, 128), ([40000, 5], None, 16, 2, 64),
    ([30000, 17, 2000, 0], [4, 4, 1, 0], 64, 8, 128), ([60000], None, 4, 4, 128)])
def test_heavy_merges(lib, cuda, monkeypatch, lengths, counts, hq, hkv, d):
    """Few requests of long contexts: units of many pieces and columns, folded
    by the merge kernel by default, give the rows that the fold inside the
    decode kernel gives - bit for bit where its weights fit its scratch (4096
    at head_dim 128) - and the oracle's."""
    b = make(lengths, counts, hq, hkv, d, torch.bfloat16, 9, cuda)
    kv = b.paged_kv, b.extra["ks"], b.extra["vs"]
    out = {}
    for merge in ("fused", "kernel", None):
        if merge:
            monkeypatch.setenv("FADECODE_MERGE", merge)
        else:
            monkeypatch.delenv("FADECODE_MERGE")
        p = plan(lib, b)
        if merge:
            assert p.info["fused_merge"] == int(merge == "fused")
        pieces = int(p.work()[2][:, 3].max())
        columns = hq // hkv * p.info["q_len"]
        if merge is None:
            assert p.info["fused_merge"] == int(pieces * columns <= 320)
        o, lse = p.run_block_scales(b.q, *kv)
        po, plse = p.run(b.q, b.paged_kv, k_scale=0.01, v_scale=0.01)
        torch.cuda.synchronize()
        assert p.check() == 0
        out[merge] = o, lse, po, plse
        if merge != "fused" or pieces * columns <= 2048:
            again = p.run_block_scales(b.q, *kv)
            assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    check(b, out[None][0], out[None][1], reference(b))
    o, lse = torch.zeros_like(out[None][0]), torch.zeros_like(out[None][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run_block_scales(b.q, *kv, out=o, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out[None][0]) and torch.equal(lse, out[None][1])
    for x, y, z in zip(out["fused"], out["kernel"], out[None]):
        assert torch.equal(y, z) or torch.equal(x, z)
        if pieces * columns <= 2048:
            assert torch.equal(x, y)


def test_many_short_requests(lib, cuda):
    """Thousands of segments of 0 to 3 pages, fresh plans, on the first launch
    right after another kernel's."""
    for seed in range(6):
        rng = np.random.default_rng(seed)
        lengths = rng.integers(0, 48, 2500)
        b = make(list(lengths), None, 64, 8, 128, torch.bfloat16, seed, cuda, spread=3.0)
        p = plan(lib, b)
        p.run(b.q, b.paged_kv)
        o, lse = run(p, b)
        assert p.check() == 0
        check(b, o, lse, reference(b))


def test_refusals(lib, cuda):
    b = make([40], None, 8, 2, 128, torch.bfloat16, 1, cuda)
    p = plan(lib, b)
    ks = b.extra["ks"]
    for bad in (ks[:-1], ks.double(), ks.cpu(), torch.ones((b.num_pages, 2, 16), device=cuda),
                torch.ones((2, b.num_pages), device=cuda).T):
        with pytest.raises(ValueError):
            p.run_block_scales(b.q, b.paged_kv, bad, ks)
        with pytest.raises(ValueError):
            p.run_block_scales(b.q, b.paged_kv, ks, bad)
    n = W.make_batch(batch_lengths=[40], num_qo_heads=8, num_kv_heads=2, head_dim=128,
                     q_dtype=torch.bfloat16, kv_dtype=torch.bfloat16, seed=1, device=cuda)
    pn = lib.plan(n.indptr, n.indices, n.last_page_len, 8, 2, 128, 16)
    pc = lib.cascade_plan(n.indices[:1], [0, 1], n.indices[1:2], [16], 8, 2, 128, 16)
    with pytest.raises(lib.FaError):
        pc.run_block_scales(n.q, n.paged_kv, *(torch.ones((n.num_pages, 2), device=cuda),) * 2)
    with pytest.raises(lib.FaError):
        pn.run_block_scales(n.q, n.paged_kv, *(torch.ones((n.num_pages, 2), device=cuda),) * 2)

"""Calls of the append and of block-scaled decode that their documentation allows:
captured, on other streams and two at once, with page-locked and broadcast
tensors and workspaces of another type.  Each against the same call in its
plain form, bit for bit."""
import pytest
import torch

from paged_kv_decode_fa_gb300 import workloads as W
from tests.test_append import BF16, E4M3, F16, F32, Batch

pytestmark = pytest.mark.gpu


def same(x, y):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x, y))


def cascade(lib, cuda, dtype=BF16):
    b = W.make_cascade_batch(prefix_pages=70, suffix_lengths=[(7 * i) % 61 for i in range(40)],
                             num_qo_heads=24, num_kv_heads=3, head_dim=128, dtype=dtype,
                             kv_dtype=E4M3, seed=3, device=cuda)
    g = torch.Generator(device=cuda).manual_seed(1)
    ks, vs = (torch.exp2(torch.randint(-8, -4, (b.num_pages, 3), generator=g, device=cuda).float())
              for _ in range(2))
    make = lambda: lib.cascade_plan(*W.cascade_parts(b), 24, 3, 128, 16, q_data_type=dtype,  # noqa: E731
                                    kv_data_type=E4M3)
    return b, ks, vs, make


@pytest.mark.parametrize("overlap", ["0", "1"])
def test_cascade_block_scales_captured_and_on_another_stream(lib, cuda, monkeypatch, overlap):
    b, ks, vs, make = cascade(lib, cuda)
    want = make().run_block_scales(b.q, b.paged_kv, ks, vs)
    torch.cuda.synchronize()
    monkeypatch.setenv("FADECODE_CASCADE_OVERLAP", overlap)
    p = make()
    o, lse = torch.zeros_like(b.q), torch.zeros(b.q.shape[:2], device=cuda)
    side = torch.cuda.Stream()
    p.run_block_scales(b.q, b.paged_kv, ks, vs, out=o, lse=lse, stream=side)
    side.synchronize()
    assert same((o, lse), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run_block_scales(b.q, b.paged_kv, ks, vs, out=o, lse=lse)
    for _ in range(3):
        o.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same((o, lse), want)
    assert p.check() == 0


def test_decode_block_scales_with_page_locked_rows(lib, cuda):
    """q, o and lse in page-locked memory, the page table too."""
    b = Batch([0] * 5, [700, 1, 16, 90, 333], 16, 4, 128, BF16, E4M3, seed=7)
    ks, vs = (torch.zeros((b.num_pages, 4), device=cuda) for _ in range(2))
    ids = b.indices.cpu().pin_memory()
    ap = lib.plan_append(b.indptr, ids, b.last, b.append, 16, 4, 128, 16, q_data_type=BF16,
                         kv_data_type=E4M3, rotary=lib.RotaryTable(128))
    ap.run_block_scales(b.k, b.v, b.kv, ks, vs)
    kv2, ks2, vs2 = b.kv.clone(), ks.clone(), vs.clone()
    b.plan(lib, lib.RotaryTable(128)).run_block_scales(b.k, b.v, kv2, ks2, vs2)
    torch.cuda.synchronize()
    assert same((b.kv, ks, vs), (kv2, ks2, vs2)) and ap.check() == 0
    kw = dict(q_data_type=BF16, kv_data_type=E4M3)
    q = torch.randn((5, 16, 128), device=cuda).to(BF16)
    want = lib.plan(b.indptr, b.indices, b.last, 16, 4, 128, 16, **kw).run_block_scales(
        q, b.kv, ks, vs)
    p = lib.plan(b.indptr, ids, b.last, 16, 4, 128, 16, **kw)
    got = p.run_block_scales(q.cpu().pin_memory(), b.kv, ks, vs)
    torch.cuda.synchronize()
    assert not got[0].is_cuda and got[0].is_pinned() and p.check() == 0
    assert same([t.to(cuda) for t in got], want)


@pytest.mark.parametrize("mode", ["native", "tensor", "head", "token", "block"])
def test_one_append_plan_on_two_streams_at_once(lib, cuda, mode):
    """The plan is only read: two caches, two streams."""
    kvt = F16 if mode == "native" else E4M3
    b = Batch([0, 5, 31, 400], [300, 1, 40, 900], 8, 2, 64, F16, kvt, seed=5)
    p = b.plan(lib, lib.RotaryTable(64, interleaved=True))
    shape = {"head": (2,), "token": (b.num_pages, 2, 16)}.get(mode, (b.num_pages, 2))

    def run(kv, ks, vs, q_out, stream):
        if mode in ("native", "tensor"):
            s = {} if mode == "native" else dict(k_scale=0.5, v_scale=0.25)
            p.run(b.k, b.v, kv, q=b.q, q_out=q_out, stream=stream, **s)
        else:
            getattr(p, f"run_{mode}_scales")(b.k, b.v, kv, ks, vs, q=b.q, q_out=q_out,
                                             stream=stream)

    states = [[b.kv.clone(), torch.full(shape, 0.5, device=cuda),
               torch.full(shape, 0.5, device=cuda), torch.empty_like(b.q.contiguous())]
              for _ in range(3)]
    run(*states[0], None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, state in zip(streams, states[1:]):
        run(*state, s)
    torch.cuda.synchronize()
    assert same(states[1], states[0]) and same(states[2], states[0])
    graph = torch.cuda.CUDAGraph()
    again = [b.kv.clone(), torch.full(shape, 0.5, device=cuda),
             torch.full(shape, 0.5, device=cuda), torch.empty_like(states[0][3])]
    with torch.cuda.graph(graph):
        run(*again, None)
    graph.replay()
    torch.cuda.synchronize()
    assert same(again, states[0])
    assert p.check() == 0


@pytest.mark.parametrize("dtype,kvt", [(F32, F32), (BF16, BF16), (F16, E4M3)])
def test_broadcast_heads_and_tokens(lib, cuda, dtype, kvt):
    """Strides of zero: one K and V for every kv head, one row for every token."""
    b = Batch([3, 0], [30, 9], 8, 4, 128, dtype, kvt, seed=2)
    rot = lib.RotaryTable(128)
    p = b.plan(lib, rot)
    for k, v in ((b.k[:, :1].expand(-1, 4, -1), b.v[:, 1:2].expand(-1, 4, -1)),
                 (b.k[:1].expand(b.T, -1, -1), b.v[:1].expand(b.T, -1, -1)),
                 (b.k[:1, :1].expand(b.T, 4, -1), b.v)):
        one, two = b.kv.clone(), b.kv.clone()
        kw = {} if kvt != E4M3 else dict(k_scale=0.25, v_scale=0.5)
        q1 = p.run(k, v, one, q=b.q[:, :1].expand(-1, 8, -1), **kw)
        q2 = p.run(k.contiguous(), v.contiguous(), two,
                   q=b.q[:, :1].expand(-1, 8, -1).contiguous(), **kw)
        torch.cuda.synchronize()
        assert same((one, q1), (two, q2))


def test_workspaces_of_another_type_and_size(lib, cuda):
    b = Batch([3, 0], [30, 9], 8, 2, 128, BF16, BF16, seed=2)
    want = b.kv.clone()
    b.plan(lib).run(b.k, b.v, want)
    for ws in (torch.empty(1 << 20, dtype=torch.int32, device=cuda),
               torch.empty(1 << 12, dtype=torch.float64, device=cuda)):
        got = b.kv.clone()
        p = b.plan(lib, workspace=ws)
        p.run(b.k, b.v, got)
        torch.cuda.synchronize()
        assert same([got], [want]) and p.check() == 0


def test_rows_that_are_padded_are_refused(lib, cuda):
    """More rows than the plan has tokens: not taken for a longer append."""
    b = Batch([3, 0], [30, 9], 8, 2, 128, BF16, BF16, seed=2)
    p = b.plan(lib)
    before = b.kv.clone()
    pad = lambda x: torch.cat([x, x[:1]])  # noqa: E731
    for k, v, q in ((pad(b.k), b.v, None), (b.k, pad(b.v), None), (b.k, b.v, pad(b.q))):
        with pytest.raises(ValueError):
            p.run(k, v, b.kv, q=q)
    torch.cuda.synchronize()
    assert same([b.kv], [before])


def test_multi_token_and_ragged_captured_with_buckets(lib, cuda, monkeypatch):
    monkeypatch.setenv("FADECODE_BUCKETS", "all")
    b = W.make_ragged_q_batch(batch_lengths=[3000, 40, 2500, 17, 1000, 611, 9],
                              q_counts=[4, 1, 3, 0, 2, 4, 1], num_qo_heads=16, num_kv_heads=2,
                              head_dim=128, q_dtype=BF16, kv_dtype=E4M3, seed=1, device=cuda)
    ks, vs = (torch.full((b.num_pages, 2), 2.0 ** -6, device=cuda) for _ in range(2))
    p = lib.plan_ragged_q(b.indptr, b.indices, b.last_page_len, b.extra["qo_indptr"], 16, 2, 128, 16,
                          q_data_type=BF16, kv_data_type=E4M3)
    assert p.info["num_buckets"] > 1
    want = p.run_block_scales(b.q, b.paged_kv, ks, vs)
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run_block_scales(b.q, b.paged_kv, ks, vs, out=o, lse=lse)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same((o, lse), want)
    assert p.check() == 0

"""Outputs and workspaces that a call on another stream makes for itself do not
come from memory that the current stream has freed and still uses."""
import pytest
import torch

from tests.test_append import BF16, E4M3, Batch

pytestmark = pytest.mark.gpu
SHAPE = (8, 2, 128, 16)


def calls(lib, cuda):
    b = Batch([60] * 64, [4] * 64, 8, 2, 128, BF16, E4M3, seed=1)
    b.kv.view(torch.uint8).bitwise_and_(0x77)   # no NaN codes
    n = b.num_pages
    ks, vs = (torch.ones((n, 2), device=cuda) for _ in range(2))
    kt, vt = (torch.ones((n, 2, 16), device=cuda) for _ in range(2))
    kw = dict(q_data_type=BF16, kv_data_type=E4M3)
    ap = b.plan(lib)
    dp = lib.plan(b.indptr, b.indices, b.last, *SHAPE, **kw)
    cp = lib.cascade_plan(b.indices[:1], b.indptr, b.indices, b.last, *SHAPE, **kw)
    q = torch.randn((64, 8, 128), device=cuda).to(BF16)
    lse = torch.randn((64, 8), device=cuda)
    head = torch.ones(2, device=cuda)
    out = lambda r: r[0]  # noqa: E731
    return {
        "append": lambda s: ap.run(b.k, b.v, b.kv, q=b.q, stream=s),
        "append block": lambda s: ap.run_block_scales(b.k, b.v, b.kv, ks, vs, q=b.q, stream=s),
        "decode": lambda s: out(dp.run(q, b.kv, stream=s)),
        "decode head": lambda s: out(dp.run_head_scales(q, b.kv, head, head, stream=s)),
        "decode token": lambda s: out(dp.run_token_scales(q, b.kv, kt, vt, stream=s)),
        "decode block": lambda s: out(dp.run_block_scales(q, b.kv, ks, vs, stream=s)),
        "cascade": lambda s: out(cp.run(q, b.kv, stream=s)),
        "cascade block": lambda s: out(cp.run_block_scales(q, b.kv, ks, vs, stream=s)),
        "merge": lambda s: out(lib.merge_states(q, lse, q, lse, stream=s)),
        "append plan": lambda s: b.plan(lib, stream=s)._workspace,
        "decode plan": lambda s: lib.plan(b.indptr, b.indices, b.last, *SHAPE, stream=s,
                                          **kw)._workspace,
        "cascade plan": lambda s: lib.cascade_plan(b.indices[:1], b.indptr, b.indices, b.last,
                                                   *SHAPE, stream=s, **kw)._keep[-1],
    }


NAMES = ["append", "append block", "decode", "decode head", "decode token", "decode block",
         "cascade", "cascade block", "merge", "append plan", "decode plan", "cascade plan"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(lib, cuda, name, raw):
    call = calls(lib, cuda)[name]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    first = call(stream)
    torch.cuda.synchronize()
    want, shape, dtype = first.clone(), first.shape, first.dtype
    del first
    # blocks of that size that the current stream frees while a copy of them waits
    held = [torch.full(shape, 1, dtype=dtype, device=cuda) for _ in range(4)]
    kept = torch.empty_like(held[0])
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for x in held:
        kept.copy_(x)
    freed = {x.data_ptr() for x in held}
    del held, x
    got = call(stream)
    assert got.data_ptr() not in freed
    side.synchronize()
    assert not torch.cuda.current_stream().query()   # the copies still wait
    torch.cuda.synchronize()
    if "plan" not in name:
        assert torch.equal(got, want)
    assert (kept == 1).all()


def test_output_is_not_reused_while_the_current_stream_reads_it(lib, cuda):
    call = calls(lib, cuda)["decode block"]
    side = torch.cuda.Stream()
    o = call(side)
    torch.cuda.synchronize()
    at, want = o.data_ptr(), o.clone()
    torch.cuda._sleep(100_000_000)
    kept = o.clone()
    del o
    again = call(side)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_the_null_handle_is_the_default_stream(lib, cuda):
    """stream=0 from within another stream: the default stream's memory (a block it
    freed is the first one to be taken again), not some new stream's."""
    call = calls(lib, cuda)["decode block"]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(40):                       # more than torch has streams to hand out
        x = torch.empty(want.shape, dtype=want.dtype, device=cuda)
        at = x.data_ptr()
        del x
        with torch.cuda.stream(side):
            got = call(0)
        assert got.data_ptr() == at
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del got
        torch.cuda.synchronize()


@pytest.mark.parametrize("forked", [False, True])
@pytest.mark.parametrize("name", ["append block", "decode block", "cascade block", "merge"])
def test_outputs_made_in_a_captured_call(lib, cuda, name, forked):
    """stream= the capturing stream, or one forked from it, without outputs."""
    call = calls(lib, cuda)[name]
    want = call(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        if forked:
            side.wait_stream(here)
        got = call(side if forked else here)
        if forked:
            here.wait_stream(side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        got.zero_()

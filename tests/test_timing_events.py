"""The timing events bracket a run as a whole: once the second has come, o and
lse are complete, also where a merge kernel folds the plan's heavy units."""
import pytest
import torch

from paged_kv_decode_fa_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("merge", ["kernel", "fused", None])
def test_after_event_covers_the_merge(lib, cuda, monkeypatch, merge):
    if merge:
        monkeypatch.setenv("FADECODE_MERGE", merge)
    else:
        monkeypatch.delenv("FADECODE_MERGE", raising=False)
    b = W.make_batch(batch_lengths=[60000, 50000], num_qo_heads=8, num_kv_heads=1, head_dim=128,
                     q_dtype=torch.bfloat16, kv_dtype=torch.bfloat16, seed=2, device=cuda)
    p = lib.plan(b.indptr, b.indices, b.last_page_len, 8, 1, 128, 16)
    assert p.info["num_merge_units"] > 0
    assert p.info["fused_merge"] == int(merge == "fused")  # a merge kernel by default
    want, want_lse = p.run(b.q, b.paged_kv)
    o, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    seen, seen_lse = torch.empty_like(o), torch.empty_like(lse)
    a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    z.record()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    p.set_timing_events(a, z)
    for _ in range(8):
        o.zero_()
        lse.zero_()
        torch.cuda._sleep(4_000_000)     # both streams' work is queued by then
        p.run(b.q, b.paged_kv, out=o, lse=lse)
        other.wait_event(z)
        with torch.cuda.stream(other):
            seen.copy_(o)
            seen_lse.copy_(lse)
        torch.cuda.synchronize()
        assert torch.equal(seen, want) and torch.equal(seen_lse, want_lse)
        assert a.elapsed_time(z) > 0
    p.set_timing_events(None, None)

"""Outputs too small for what a run writes are refused, as are tensors of
another device by the block-scaled run."""
import pytest
import torch

from tests.test_append import BF16, E4M3, Batch

pytestmark = pytest.mark.gpu
SHAPE = (8, 2, 128, 16)


def runs(lib, cuda):
    b = Batch([60] * 4, [4] * 4, 8, 2, 128, BF16, E4M3, seed=1)
    n = b.num_pages
    ks, vs = (torch.ones((n, 2), device=cuda) for _ in range(2))
    kt, vt = (torch.ones((n, 2, 16), device=cuda) for _ in range(2))
    kw = dict(q_data_type=BF16, kv_data_type=E4M3)
    dp = lib.plan(b.indptr, b.indices, b.last, *SHAPE, **kw)
    cp = lib.cascade_plan(b.indices[:1], b.indptr, b.indices, b.last, *SHAPE, **kw)
    q = torch.randn((4, 8, 128), device=cuda).to(BF16)
    head = torch.ones(2, device=cuda)
    return q, {
        "run": lambda **o: dp.run(q, b.kv, **o),
        "head": lambda **o: dp.run_head_scales(q, b.kv, head, head, **o),
        "token": lambda **o: dp.run_token_scales(q, b.kv, kt, vt, **o),
        "block": lambda **o: dp.run_block_scales(q, b.kv, ks, vs, **o),
        "cascade": lambda **o: cp.run(q, b.kv, **o),
        "cascade block": lambda **o: cp.run_block_scales(q, b.kv, ks, vs, **o),
    }


@pytest.mark.parametrize("name", ["run", "head", "token", "block", "cascade", "cascade block"])
def test_small_outputs_are_refused(lib, cuda, name):
    q, all_runs = runs(lib, cuda)
    run = all_runs[name]
    # views into larger buffers: an unmended run writes past the view, inside the buffer
    big, big_lse = torch.zeros((8, 8, 128), dtype=BF16, device=cuda), torch.zeros((8, 8), device=cuda)
    for kw in (dict(out=big[:3]), dict(out=big.view(-1)[:q.numel() - 1]),
               dict(lse=big_lse[:3]), dict(lse=big_lse.view(-1)[:31]),
               dict(lse=big_lse.view(BF16).view(-1)[:32].view(4, 8))):
        with pytest.raises(ValueError):
            run(**kw)
    torch.cuda.synchronize()
    assert not big.any() and not big_lse.any()
    o, lse = run(out=big, lse=big_lse)         # room to spare is not refused
    want, want_lse = run()
    torch.cuda.synchronize()
    assert torch.equal(big[:4].view(torch.int16), want.view(torch.int16))
    assert torch.equal(big_lse[:4].view(torch.int32), want_lse.view(torch.int32))
    assert not big[4:].any() and not big_lse[4:].any()


def test_block_scales_on_another_device_are_refused(lib, cuda, monkeypatch):
    q, all_runs = runs(lib, cuda)

    class Elsewhere(torch.Tensor):
        """A tensor that says it is on the next device."""
        def get_device(self):
            return super().get_device() + 1

    out = torch.zeros_like(q).as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        all_runs["block"](out=out)
    with pytest.raises(ValueError):
        all_runs["block"](lse=torch.zeros((4, 8), device=cuda).as_subclass(Elsewhere))

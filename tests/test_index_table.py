"""A page table shorter than indptr asks for is refused by every plan: the
kernels would read past it, and an append write wherever that points."""
import pytest
import torch

SHAPE = (8, 2, 128, 16)
CALLS = {
    "plan": lambda fa, ids: fa.plan([0, 1, 3], ids, [4, 5], *SHAPE),
    "multi_token": lambda fa, ids: fa.plan_multi_token([0, 1, 3], ids, [4, 5], 2, *SHAPE),
    "ragged_q": lambda fa, ids: fa.plan_ragged_q([0, 1, 3], ids, [4, 5], [0, 1, 2], *SHAPE),
    "cascade": lambda fa, ids: fa.cascade_plan(torch.zeros_like(ids), [0, 1, 3], ids, [4, 5],
                                               *SHAPE),
    "append": lambda fa, ids: fa.plan_append([0, 1, 3], ids, [4, 5], [0, 1, 2], *SHAPE),
    "append_tensors": lambda fa, ids: fa.plan_append(
        torch.tensor([0, 1, 3], dtype=torch.int32), ids, torch.tensor([4, 5], dtype=torch.int32),
        torch.tensor([0, 1, 2], dtype=torch.int32), *SHAPE),
}


@pytest.mark.parametrize("call", [c for c in CALLS if c != "cascade"])
def test_short_table_is_refused_before_any_cuda_call(lib, monkeypatch, call):
    monkeypatch.setattr(lib, "_reachable", lambda t: True)
    for n in (0, 2):
        with pytest.raises(ValueError, match="indptr asks for 3"):
            CALLS[call](lib, torch.zeros(n, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("call", list(CALLS))
def test_short_table(lib, cuda, call):
    for n in (1, 2):
        with pytest.raises(ValueError, match="indptr asks for 3"):
            CALLS[call](lib, torch.zeros(n, dtype=torch.int32, device=cuda))
    CALLS[call](lib, torch.zeros(3, dtype=torch.int32, device=cuda))
    CALLS[call](lib, torch.zeros(5, dtype=torch.int32, device=cuda))

"""Host arrays of a plan that int32 does not hold are refused by name."""
import numpy as np
import pytest
import torch


def test_budgets_that_do_not_fit_are_refused(lib):
    """A budget beyond 32 bits, or no whole number, is named; not cut to what fits."""
    def plan(keep, recent=0, indptr=(0, 1)):
        lib.plan_evict(np.asarray(indptr), torch.zeros(1, dtype=torch.int32), np.array([5], np.int32),
                       keep, 2, 64, 16, recent=recent)

    for big in (2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5):
        for v in (big, [big], np.array([big]), torch.tensor([big])):
            with pytest.raises(ValueError, match="keep and recent|32 bits"):
                plan(v)
            with pytest.raises(ValueError, match="keep and recent|32 bits"):
                plan(3, recent=v)
    for v in (2.5, [2.5], torch.tensor([0.5])):
        with pytest.raises(ValueError, match="keep and recent|32 bits|whole"):
            plan(v)
    with pytest.raises(ValueError, match="32 bits"):
        plan(3, indptr=np.array([0, 2 ** 32 + 1]))


def test_whole_numbers_of_any_type_are_taken(lib):
    want = np.array([0, 3, 2 ** 31 - 1], np.int32)
    for given in ([0, 3, 2 ** 31 - 1], want.astype(np.int64), want.astype(np.float64), want[::-1][::-1],
                  torch.from_numpy(want).long(), torch.from_numpy(want), want.astype(np.uint64), tuple(want)):
        got = lib._host_i32(given)
        assert got.dtype == np.int32 and got.flags.c_contiguous and np.array_equal(got, want)
    for bad in ([0, 2 ** 31], [0, 2 ** 70], [0.5], [float("nan")], torch.tensor([float("inf")]),
                np.array([2 ** 63], np.uint64), torch.tensor([-2 ** 31 - 1])):
        with pytest.raises(ValueError, match="32 bits"):
            lib._host_i32(bad)
    with pytest.raises(ValueError, match="32 bits"):
        lib.RotaryTable(32, axes=[2 ** 32] * 16)

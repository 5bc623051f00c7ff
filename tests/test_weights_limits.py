"""What one request may ask of the weights' kernels: refused on the host."""
import ctypes

import numpy as np
import pytest


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("before", [0, 3])
def test_too_many_columns_are_refused(lib, group, before):
    """A job passes through all columns of its request while other warps wait for it:
    2^26 at most.  Refused before any CUDA call; the addresses are never read."""
    arr = lambda v: np.array(v, np.int32)  # noqa: E731
    indptr, last, qo = arr((0, 1, 2)), arr((3, 3)), arr((0, before, before + 2 ** 26 // group + 1))
    out = ctypes.c_void_p()
    for q, kv in ((1, 1), (2, 2), (1, 3), (2, 3)):
        assert lib.library().fa_weights_plan(
            indptr.ctypes.data, 256, last.ctypes.data, qo.ctypes.data, 2, 2 * group, 2, 64, 16, q, kv, 256,
            1 << 20, None, ctypes.byref(out)) == -2
        assert not out.value

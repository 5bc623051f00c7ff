"""Append with positions on several axes (RotaryTable(axes=), plan_append(positions=))
against the definition in 64 bits: pair j of a token turns by its position on axis
axes[j].  Tolerances as in test_append.py: the stored type's rounding, and the
rotation's fp32 error of ROT times the pair."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_append import BF16, E4M3, F16, F32, ROT, Batch, close, code_close, f64

LENGTHS = [([0, 5, 15, 16, 31, 0, 40], [1, 0, 1, 2, 37, 9, 16]), ([0], [1]), ([33], [70])]


def rotate_axes(x, positions, rotary):
    """x [T, H, D] float64, positions [axes, T]; the bound of its fp32 error."""
    y, slack = x.copy(), np.zeros_like(x)
    for j, axis in enumerate(rotary.axes):
        a = positions[axis].astype(np.float64) * rotary.inv_freq[j]
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        i, k = (2 * j, 2 * j + 1) if rotary.interleaved else (j, j + rotary.rotary_dim // 2)
        y[..., i] = x[..., i] * c - x[..., k] * s
        y[..., k] = x[..., k] * c + x[..., i] * s
        slack[..., i] = slack[..., k] = ROT * (np.abs(x[..., i]) + np.abs(x[..., k]))
    return y, slack


def far_rotate_axes(x, positions, rotary):
    """The same for positions whose float64 angle would lose digits: reduced
    modulo a turn in integers of 2^-80 turns."""
    turns = [int(round(f * 2 ** 40)) for f in rotary.inv_freq]  # inv_freq are k 2^-40 turns * 2 pi
    y = x.copy()
    for j, axis in enumerate(rotary.axes):
        frac = np.array([(int(p) * turns[j]) % 2 ** 40 / 2 ** 40 for p in positions[axis]])
        y_c, y_s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
        k = j + rotary.rotary_dim // 2
        y[..., j] = x[..., j] * y_c - x[..., k] * y_s
        y[..., k] = x[..., k] * y_c + x[..., j] * y_s
    return y


def check(b, q, positions, rotary, scales=None):
    """The rows of q and of the pages against the definition."""
    want, slack = rotate_axes(f64(b.q), positions, rotary)
    close(f64(q), want, slack, b.q_dtype)
    k, ks = rotate_axes(f64(b.k), positions, rotary)
    v = f64(b.v)
    kv = f64(b.kv.float() if b.kv_dtype == E4M3 else b.kv)
    for _, row, page, slot, _ in b.places():
        if scales is None:
            close(kv[page, 0, slot], k[row], ks[row], b.q_dtype)
            close(kv[page, 1, slot], v[row], 0 * v[row], b.q_dtype)
        else:
            code_close(kv[page, 0, slot], k[row] / scales, (ks[row] + 2e-7 * abs(k[row])) / scales)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("dtype,d,hq,hkv,rotary_dim,interleaved,num_axes", [
    (F32, 64, 3, 3, 64, False, 3), (BF16, 128, 32, 8, 128, False, 3), (F16, 64, 8, 2, 48, True, 2),
    (BF16, 128, 5, 5, 16, False, 3), (F32, 128, 8, 1, 128, True, 5), (BF16, 64, 16, 4, 64, False, 1)])
def test_native(lib, cuda, dtype, d, hq, hkv, rotary_dim, interleaved, num_axes, lengths):
    b = Batch(*LENGTHS[lengths], hq, hkv, d, dtype, dtype, seed=lengths)
    rng = np.random.default_rng(5)
    axes = rng.integers(0, num_axes, rotary_dim // 2)
    axes[0] = num_axes - 1
    rotary = lib.RotaryTable(rotary_dim, axes=axes, interleaved=interleaved)
    pos = rng.integers(-3000, 5000, (num_axes, b.T)).astype(np.int32)
    p = b.plan(lib, rotary, positions=torch.from_numpy(pos).cuda())
    q = p.run(b.k, b.v, b.kv, q=b.q)
    check(b, q, pos, rotary)
    assert p.check() == 0


@pytest.mark.gpu
def test_equal_axes_are_the_ordinary_rotation(lib, cuda):
    """A text token's axes advance together: bit for bit one position's rotation."""
    b = Batch([3, 0, 200], [20, 1, 9], 16, 4, 128, BF16, BF16, seed=2)
    q0 = b.plan(lib, lib.RotaryTable(128)).run(b.k, b.v, b.kv, q=b.q)
    kv0 = b.kv.clone()
    pos = torch.tensor([[t for _, _, _, _, t in b.places()]] * 3, dtype=torch.int32, device=cuda)
    rotary = lib.RotaryTable(128, axes=np.repeat([0, 1, 2], [16, 24, 24]))
    q1 = b.plan(lib, rotary, positions=pos).run(b.k, b.v, b.kv, q=b.q)
    assert torch.equal(q0, q1) and torch.equal(kv0, b.kv)


@pytest.mark.gpu
def test_extreme_positions(lib, cuda):
    """Any int32: the angle is reduced modulo a turn in integers.  inv_freq is a whole
    number of 2^-40 turns, at most 2^-3, times 2 pi: off by 2^-53 of itself for the
    product and 2^-54.5 for the double nearest 2 pi, 2^31 positions away
    2^28 (2^-53 + 2^-54.5) turns or 2.6e-7 radians.  (The plan's own 2^-64 of a turn
    is 2^-33 there: nothing beside that.)"""
    b = Batch([0], [6], 4, 2, 64, F32, F32, seed=4)
    rng = np.random.default_rng(0)
    turns = rng.integers(1, 2 ** 37, 32)
    rotary = lib.RotaryTable(64, inv_freq=turns / 2.0 ** 40 * (2 * np.pi),
                             axes=np.arange(32) % 2)
    pos = np.array([[2 ** 31 - 1, -2 ** 31, 0, -1, 2 ** 30, 7], [-2 ** 31, 2 ** 31 - 1, -7, 1, 3, 5]],
                   np.int32)
    q = b.plan(lib, rotary, positions=torch.from_numpy(pos).cuda()).run(b.k, b.v, b.kv, q=b.q)
    rotary.inv_freq = turns / 2.0 ** 40
    want = far_rotate_axes(f64(b.q), pos, rotary)
    x = np.abs(f64(b.q))
    size = np.concatenate([x[..., :32] + x[..., 32:]] * 2, -1)
    close(f64(q), want, (ROT + 2.6e-7) * size, F32)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["head", "token", "block"])
def test_e4m3(lib, cuda, mode):
    b = Batch(*LENGTHS[0], 16, 4, 128, BF16, E4M3, seed=6)
    rng = np.random.default_rng(1)
    rotary = lib.RotaryTable(128, axes=np.arange(64) % 3)
    pos = rng.integers(0, 900, (3, b.T)).astype(np.int32)
    p = b.plan(lib, rotary, positions=torch.from_numpy(pos).cuda())
    if mode == "head":
        ks = torch.tensor([0.02, 0.03, 0.05, 0.5], device=cuda)
        q = p.run_head_scales(b.k, b.v, b.kv, ks, ks.clone(), q=b.q)
        return check(b, q, pos, rotary, f64(ks)[:, None])
    shape = (b.num_pages, 4, 16) if mode == "token" else (b.num_pages, 4)
    ks = torch.zeros(shape, device=cuda)
    vs = torch.zeros(shape, device=cuda)
    run = p.run_token_scales if mode == "token" else p.run_block_scales
    q = run(b.k, b.v, b.kv, ks, vs, q=b.q)
    want, slack = rotate_axes(f64(b.q), pos, rotary)
    close(f64(q), want, slack, BF16)
    k, slack = rotate_axes(f64(b.k), pos, rotary)
    kv = f64(b.kv.float())
    for _, row, page, slot, _ in b.places():
        s = f64(ks)[page, :, slot] if mode == "token" else f64(ks)[page]
        code_close(kv[page, 0, slot], k[row] / s[:, None],
                   (slack[row] + 2e-7 * np.abs(k[row])) / s[:, None])


@pytest.mark.gpu
def test_positions_are_read_by_each_run(lib, cuda):
    """A captured run replayed after its positions were written anew."""
    b = Batch([0, 9, 30], [1, 1, 1], 8, 2, 128, BF16, BF16, seed=9)
    rotary = lib.RotaryTable(128, axes=np.arange(64) % 3)
    pos = torch.tensor([[1, 2, 3], [4, 5, 6], [7, 8, 9]], dtype=torch.int32, device=cuda)
    p = b.plan(lib, rotary, positions=pos)
    q = torch.empty_like(b.q.contiguous())
    p.run(b.k, b.v, b.kv, q=b.q, q_out=q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(b.k, b.v, b.kv, q=b.q, q_out=q)
    new = np.array([[100, 7, 0], [3, 900, 12], [55, 1, 31]], np.int32)
    pos.copy_(torch.from_numpy(new))
    graph.replay()
    torch.cuda.synchronize()
    check(b, q, new, rotary)


@pytest.mark.gpu
def test_nothing_to_append(lib, cuda):
    b = Batch([5, 0], [0, 0], 8, 2, 64, BF16, BF16)
    rotary = lib.RotaryTable(64, axes=np.arange(32) % 3)
    pos = torch.empty((3, 0), dtype=torch.int32, device=cuda)
    before = b.kv.clone()
    q = b.plan(lib, rotary, positions=pos).run(b.k, b.v, b.kv, q=b.q)
    assert q.shape == (0, 8, 64) and torch.equal(b.kv, before)


# ---------------------------------------------------------------- refusals

def host_plan(lib, *, positions=256, num_axes=3, axis=(0,) * 7 + (2,), rotary=16, d=128, append=(0, 2),
              axis_null=False):
    """fa_append_plan_axes with addresses that no refused call touches."""
    arr = lambda v: np.array(v, np.int32)  # noqa: E731
    ptr, last, app, ax = arr((0, 1)), arr((3,)), arr(append), arr(axis)
    f = np.ones(max(rotary // 2, 1))
    out = ctypes.c_void_p()
    rc = lib.library().fa_append_plan_axes(
        ptr.ctypes.data, 256, last.ctypes.data, app.ctypes.data, positions, num_axes,
        None if axis_null else ax.ctypes.data, 1, 8, 2, d, 16, 1, 1, f.ctypes.data, rotary, 0, 256,
        256, None, ctypes.byref(out))
    assert not out.value
    return rc


def test_plan_refusals(lib):
    invalid, unsupported, small = -1, -2, -3
    for kw, rc in [(dict(positions=None), invalid), (dict(positions=258), invalid),
                   (dict(num_axes=0), invalid), (dict(num_axes=2), invalid),
                   (dict(axis=(-1,) * 8), invalid), (dict(axis_null=True), invalid),
                   (dict(rotary=0), invalid), (dict(rotary=144, axis=(0,) * 72), invalid),
                   (dict(rotary=8), unsupported), (dict(append=(0, 4)), invalid),
                   (dict(d=96), unsupported), (dict(), small)]:
        assert host_plan(lib, **kw) == rc, kw


def test_table_refusals(lib):
    t = lib.RotaryTable(32, axes=[0] * 8 + [2] * 8)
    assert t.num_axes == 3 and lib.RotaryTable(32).axes is None
    for bad in ([0] * 15, [-1] + [0] * 15, np.zeros((2, 8))):
        with pytest.raises(ValueError):
            lib.RotaryTable(32, axes=bad)


@pytest.mark.gpu
def test_position_refusals(lib, cuda):
    b = Batch([0, 5], [4, 2], 8, 2, 128, BF16, BF16, seed=1)
    rotary = lib.RotaryTable(128, axes=np.arange(64) % 3)
    good = torch.zeros((3, b.T), dtype=torch.int32, device=cuda)
    for kw in ({}, {"positions": good.long()}, {"positions": good[:2]}, {"positions": good[0]},
               {"positions": good.cpu()}, {"positions": good[:, :-1]},
               {"positions": torch.zeros((b.T, 3), dtype=torch.int32, device=cuda).T},
               {"positions": good, "offset": [0, 0]}):
        with pytest.raises(ValueError):
            b.plan(lib, rotary, **kw)
    with pytest.raises(ValueError):
        b.plan(lib, lib.RotaryTable(128), positions=good)
    with pytest.raises(ValueError):
        b.plan(lib, None, positions=good)
    b.plan(lib, rotary, positions=torch.zeros((4, b.T), dtype=torch.int32, device=cuda))

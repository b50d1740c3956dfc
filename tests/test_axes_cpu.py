"""Rotary plans of several axes, and the refusals of the calls that take them, as far as they need no GPU."""

import copy
import ctypes
import pickle

import numpy as np
import pytest

import certified_quantized_kv_gb300 as kvq
import _paged as P

ADDR = 1 << 20   # an address that is never read


def axis_table(axes, order):
    """[(axis, number within the axis)] of every pair, from the words of the definition."""
    if order == "blocks":
        return [(a, j) for a, n in enumerate(axes) for j in range(n)]
    out, done = [], [0] * len(axes)
    while len(out) < sum(axes):
        for a, n in enumerate(axes):
            if done[a] < n:
                out.append((a, done[a]))
                done[a] += 1
    return out


def frequencies(axes, order, freq, **kw):
    table = axis_table(axes, order)
    if freq == "shared":
        return P.frequencies(2 * sum(axes), **kw)
    own = [P.frequencies(2 * n, **kw) for n in axes]
    return np.array([own[a][j] for a, j in table])


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts", "yarn"])
@pytest.mark.parametrize("axes,order,freq", [((16, 24, 24), "blocks", "shared"), ((24, 20, 20), "cycled", "shared"),
                                             ((8, 28, 28), "blocks", "own"), ((3, 2, 9, 5), "cycled", "own"), ((32,), "cycled", "own")])
def test_plan(axes, order, freq, scaling):
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, original_ctx=8192, low=1.0, high=4.0)
    n = sum(axes)
    plan = kvq.RopePlan(128, rotary_dim=2 * n, axes=axes, axis_order=order, axis_frequencies=freq, **kw)
    w = frequencies(axes, order, freq, **kw)
    got = np.array([int(s) for s in plan.plan.step[:n]], np.float64) / 2.0 ** 64 * 2 * np.pi
    assert np.all(np.abs(got - w) <= 2.0 ** -48 * w + 2.0 ** -60)
    assert not any(plan.plan.step[n:]) and not any(s & 3 for s in plan.plan.step)
    assert list(plan.whole.axis[:n]) == [a for a, _ in axis_table(axes, order)] and plan.n_axes == len(axes)


def test_dealt_in_turn():
    plan = kvq.RopePlan(128, axes=(24, 20, 20), axis_order="cycled")
    assert list(plan.whole.axis[:64]) == [0, 1, 2] * 20 + [0] * 4


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))])
def test_copies_hold_their_own_struct(again):
    plan = kvq.RopePlan(128, axes=(16, 24, 24))
    steps, axis, at = list(plan.plan.step), list(plan.whole.axis), plan.address
    other = again(plan)
    ctypes.memset(at, 0, ctypes.sizeof(plan.whole))
    assert other.n_axes == 3 and other.address == ctypes.addressof(other.whole) == ctypes.addressof(other.plan) != at
    assert list(other.plan.step) == steps and list(other.whole.axis) == axis


def _init(axes=(16, 24, 24), order=0, own=0, n=None, **kw):
    cfg = dict(head_dim=128, rotary_dim=128, interleaved=0, scaling=0, base=10000.0, factor=1.0, original_ctx=0,
               low=1.0, high=32.0, magnitude=0.0)
    cfg.update(kw)
    c, p = kvq.kvq_rope_config(**cfg), kvq.kvq_rope_axes_plan()
    pairs = (ctypes.c_int32 * len(axes))(*axes) if axes is not None else None
    return kvq.load_library().kvq_rope_axes_plan_init(ctypes.byref(c), len(axes or ()) if n is None else n, pairs, order, own,
                                                      ctypes.byref(p)), p


@pytest.mark.parametrize("bad,word", [
    (dict(axes=()), b"n_axes"), (dict(axes=(16, 16, 16, 8, 8)), b"n_axes"), (dict(axes=(16, 24, 25)), b"rotary_dim / 2"),
    (dict(axes=(0, 32, 32)), b"pair at least"), (dict(axes=(-8, 40, 32)), b"pair at least"), (dict(axes=(2 ** 31 - 1, 2 ** 31 - 1, 66)), b"rotary_dim / 2"),
    (dict(order=2), b"order"), (dict(own=2), b"own_frequencies"), (dict(head_dim=127), b"head_dim"), (dict(base=1.0), b"base"),
    (dict(axes=None, n=3), b"NULL"), (dict(axes=(1, 63), own=1, scaling=2, factor=2.0), b"NTK"),
])
def test_plan_refusals(bad, word):
    st, p = _init(**bad)
    assert st == kvq.KVQ_ERR_INVALID and word in kvq.load_library().kvq_last_error()
    assert p.n_axes == 0 and not any(p.plan.step)       # left as it was


def test_plan_refusals_in_python():
    with pytest.raises(ValueError):
        kvq.RopePlan(128, axes=(32, 32), axis_order="other")
    with pytest.raises(ValueError):
        kvq.RopePlan(128, axes=(32, 32), axis_frequencies="other")
    with pytest.raises(kvq.KvqError):
        kvq.RopePlan(128, axes=(32, 33))
    with pytest.raises(TypeError):
        kvq.RopePlan(128, axes=(32.0, 32.0))


def test_call_refusals():
    """Checks that come before the first CUDA call."""
    lib = kvq.load_library()
    _, plan = _init()

    def rope(p=plan, stride=4, x=ADDR, T=4, dtype=0):
        return lib.kvq_rope_axes(ctypes.byref(p) if p is not None else None, dtype, x, 256, 128, ADDR, stride, T, 2, ADDR, 256, 128, None)

    def append(p=plan, stride=4, pos=ADDR, T=4, hd=128):
        return lib.kvq_paged_append_axes(ctypes.byref(p) if p is not None else None, 0, ADDR, 256, 128, ADDR, 256, 128, ADDR, pos, stride,
                                         T, 2, hd, ADDR, 3, None, 0, 0, 0, None, 0, 0, None)

    none = kvq.kvq_rope_axes_plan()
    far = _init()[1]
    far.axis[3] = 3
    five = _init()[1]
    five.n_axes = 5
    for call in (rope, append):
        for kw in (dict(p=None), dict(p=none), dict(p=far), dict(p=five), dict(stride=-1)):
            assert call(**kw) == kvq.KVQ_ERR_INVALID, kw
            assert call.__name__.encode() + b"_axes:" in lib.kvq_last_error()
        assert call(T=0) == kvq.KVQ_OK
    assert append(pos=None) == kvq.KVQ_ERR_INVALID and append(hd=64) == kvq.KVQ_ERR_INVALID
    assert rope(dtype=2) == kvq.KVQ_ERR_INVALID

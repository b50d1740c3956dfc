"""Rotary positions with several axes on the GPU, alone and within the append, against their definition in 64 bits
and against the calls of one axis.  Tolerances as in test_gpu_paged.py: the axis only says which position enters."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402
from test_axes_cpu import axis_table, frequencies  # noqa: E402
from test_gpu_paged import HALF, ROPES, TINY, TYPES, _append_case, _check_append, _f64, _gen, _ints, _randn  # noqa: E402


def _positions(n_axes, T, seed, far=2000000):
    return torch.randint(-far, far, (n_axes, T), generator=_gen(seed)).int().cuda()


def _turned(x, pos, axes, order, freq, inter, kw):
    """[T, H, D] float64 turned pair by pair."""
    w, m = frequencies(axes, order, freq, **kw), 1.0
    if kw.get("scaling") == "yarn":
        m = 0.1 * np.log(kw["factor"]) + 1
    rd, y, p = 2 * sum(axes), np.array(x), pos.cpu().numpy().astype(np.float64)
    for i, (a, _) in enumerate(axis_table(axes, order)):
        i0, i1 = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
        c, s = np.cos(p[a] * w[i])[:, None] * m, np.sin(p[a] * w[i])[:, None] * m
        y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i1] * c + x[..., i0] * s
    return y, m


def _check(got, x, pos, axes, order, freq, inter, kw):
    rd, xf = 2 * sum(axes), _f64(x)
    ref, m = _turned(xf, pos, axes, order, freq, inter, kw)
    i0, i1 = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, rd // 2), slice(rd // 2, rd))
    both = np.zeros_like(xf)
    both[..., i0] = both[..., i1] = np.abs(xf[..., i0]) + np.abs(xf[..., i1])
    tol = np.abs(ref) * HALF[x.dtype] + TINY[x.dtype] + both * m * 2.0 ** -21 * (1 + HALF[x.dtype])
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= tol), float((err - tol).max())
    assert torch.equal(got[..., rd:], x[..., rd:])


CASES = [(1, 1, 128, (16, 24, 24), "blocks", "shared", 0), (67, 3, 64, (7, 9, 16), "cycled", "own", 1),
         (33, 5, 128, (4, 3, 3, 3), "cycled", "shared", 4), (130, 7, 96, (8, 20, 20), "blocks", "own", 2),
         (9, 2, 8, (1, 1), "blocks", "shared", 0), (3, 1, 256, (64, 64), "cycled", "own", 3),
         (301, 9, 80, (16,), "blocks", "shared", 4), (1000, 33, 64, (8, 8, 8), "cycled", "shared", 0),
         (70, 2, 136, (20, 36), "blocks", "own", 1), (5000, 3, 128, (10, 5, 11), "blocks", "shared", 0)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,axes,order,freq,kind", CASES)
def test_rope(T, H, D, axes, order, freq, kind, layout, dt):
    kw = ROPES[kind]
    plan = kvq.RopePlan(D, rotary_dim=2 * sum(axes), layout=layout, axes=axes, axis_order=order, axis_frequencies=freq, **kw)
    x, pos = _randn((T, H, D), dt, T + D), _positions(len(axes), T, H)
    wide = torch.full((T, H + 1, D + 8), 3.0, dtype=dt, device="cuda")
    out = kvq.rope(x, pos, plan, out=wide[:, :H, :D])
    _check(out, x, pos, axes, order, freq, layout == "interleaved", kw)
    assert (wide[:, H] == 3).all() and (wide[..., D:] == 3).all()
    same = x.clone()
    assert kvq.rope(same, pos, plan, out=same) is same and torch.equal(same, out)


def test_extreme_positions():
    """Frequencies in double agree to 2^-48 relative: 2^31 positions turn that into 2^-17 rad."""
    pos = _ints([[0, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1], [-1, 5, 123456789, -2 ** 31], [2 ** 31 - 1, 0, 1, -7]])
    x = _randn((4, 2, 128), torch.float16, 3)
    for order in ("blocks", "cycled"):
        plan = kvq.RopePlan(128, base=500000.0, axes=(16, 24, 24), axis_order=order)
        ref, _ = _turned(_f64(x), pos, (16, 24, 24), order, "shared", False, dict(base=500000.0))
        assert np.abs(_f64(kvq.rope(x, pos, plan)) - ref).max() <= 8 * (2.0 ** -11 + 2.0 ** -16)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [128, 52, 36, 8])
def test_one_position_on_every_axis_is_the_call_of_one_axis(layout, rd):
    """Bit for bit, also with an axis stride of 0, and with positions of rows that are further apart."""
    n, T = rd // 2, 77
    one = kvq.RopePlan(128, rotary_dim=rd, layout=layout, **ROPES[3])
    plan = kvq.RopePlan(128, rotary_dim=rd, layout=layout, axes=(1, n - 3, 2), axis_order="cycled", **ROPES[3])
    x, pos = _randn((T, 5, 128), torch.bfloat16, rd), _positions(1, T, 4)
    want = kvq.rope(x, pos[0], one)
    assert torch.equal(kvq.rope(x, pos.expand(3, T), plan), want)
    apart = torch.zeros(3, T + 9, dtype=torch.int32, device="cuda")
    apart[:, :T] = pos
    assert torch.equal(kvq.rope(x, apart[:, :T], plan), want)
    pages = [torch.zeros(2, 5, kvq.paged_page_bytes(128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.arange(T).int().cuda()
    q = [torch.empty_like(x) for _ in range(2)]
    kvq.paged_append(pages[0], x, x, slots, positions=pos[0], plan=one, q=x, q_out=q[0])
    kvq.paged_append(pages[1], x, x, slots, positions=apart[:, :T], plan=plan, q=x, q_out=q[1])
    assert torch.equal(pages[0], pages[1]) and torch.equal(q[0], q[1])


def test_the_transpose_is_the_gradient():
    """<R(p) x, y> = <x, R(-p) y>, two roundings of 2^-11 against sum |x_i| |y_i|."""
    T, H, D = 11, 3, 128
    plan = kvq.RopePlan(D, axes=(24, 20, 20), axis_order="cycled")
    x, y, pos = _randn((T, H, D), torch.float16, 1), _randn((T, H, D), torch.float16, 2), _positions(3, T, 5)
    a = (_f64(kvq.rope(x, pos, plan)) * _f64(y)).sum(-1)
    b = (_f64(x) * _f64(kvq.rope(y, -pos, plan))).sum(-1)
    assert np.all(np.abs(a - b) <= 2 * 2.0 ** -11 * np.abs(_f64(x)).sum(-1) * np.abs(_f64(y)).max(-1) + 2.0 ** -10)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,Hq,Hkv,D,axes,order,freq,layout,kind", [
    (64, 8, 2, 128, (16, 24, 24), "blocks", "shared", "half", 3), (131, 0, 3, 64, (8, 12, 12), "cycled", "own", "interleaved", 0),
    (77, 5, 5, 128, (9, 8, 9), "cycled", "shared", "half", 1), (40, 4, 1, 64, (6, 7), "blocks", "own", "half", 0),
    (1, 32, 8, 128, (24, 20, 20), "cycled", "shared", "half", 0), (300, 6, 2, 128, (5, 5, 5, 5), "blocks", "shared", "interleaved", 0)])
def test_append(T, Hq, Hkv, D, axes, order, freq, layout, kind, dt):
    kw = ROPES[kind]
    k, v, slots, _, pages = _append_case(T, Hkv, D, dt, T)
    pos = _positions(len(axes), T, T + 1, far=200000)
    plan = kvq.RopePlan(D, rotary_dim=2 * sum(axes), layout=layout, axes=axes, axis_order=order, axis_frequencies=freq, **kw)
    before = pages.clone()
    q = _randn((T, Hq, D), dt, 9) if Hq else None
    q_out = torch.empty_like(q) if Hq else None
    kvq.paged_append(pages, k, v, slots, positions=pos, plan=plan, q=q, q_out=q_out)
    turned, m = _turned(_f64(k), pos, axes, order, freq, layout == "interleaved", kw)
    _check_append(before, pages, turned, _f64(v), slots, D, key_err=2.0 ** -21 * 2 * np.abs(_f64(k)).max() * m)
    if Hq:
        assert torch.equal(q_out, kvq.rope(q, pos, plan))
        same = q.clone()
        kvq.paged_append(pages, k, v, slots, positions=pos, plan=plan, q=same, q_out=same)
        assert torch.equal(same, q_out)


def test_refusals():
    plan, one = kvq.RopePlan(128, axes=(32, 32)), kvq.RopePlan(128)
    x, pos = torch.zeros(4, 2, 128, dtype=torch.float16, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    pages = torch.zeros(1, 2, kvq.paged_page_bytes(128), dtype=torch.uint8, device="cuda")
    slots = _ints([0, 1, 2, 3])
    for p, bad in ((plan, pos[0]), (plan, pos[:1]), (plan, pos.long()), (plan, pos.cpu()), (plan, pos[:, :3]), (one, pos),
                   (plan, pos.t().contiguous().t())):
        with pytest.raises(ValueError):
            kvq.rope(x, bad, p)
        with pytest.raises(ValueError):
            kvq.paged_append(pages, x, x, slots, positions=bad, plan=p)
    host = torch.zeros(2, 4, dtype=torch.int32)
    st = kvq.load_library().kvq_rope_axes(plan.address, 0, x.data_ptr(), 256, 128, host.data_ptr(), 4, 4, 2, x.data_ptr(), 256, 128, None)
    assert st == kvq.KVQ_ERR_INVALID
    torch.cuda.synchronize()

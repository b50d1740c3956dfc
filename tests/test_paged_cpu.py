"""Rotary plans, the page layout and the refusals of the paged 4-bit cache's calls, as far
as they need no GPU: every check tested here runs before the first CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import certified_quantized_kv_gb300 as kvq
import _paged as P


def _plan(**kw):
    cfg = dict(head_dim=128, rotary_dim=128, interleaved=0, scaling=0, base=10000.0, factor=1.0, original_ctx=0,
               low=1.0, high=32.0, magnitude=0.0)
    cfg.update(kw)
    c, p = kvq.kvq_rope_config(**cfg), kvq.kvq_rope_plan()
    return kvq.load_library().kvq_rope_plan_init(ctypes.byref(c), ctypes.byref(p)), p


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts", "yarn"])
@pytest.mark.parametrize("rd", [4, 26, 64, 128, 256])
def test_plan_frequencies(scaling, rd):
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, original_ctx=8192, low=1.0, high=4.0)
    plan = kvq.RopePlan(256, rotary_dim=rd, **kw)
    w = P.frequencies(rd, **kw)
    got = np.array([int(s) for s in plan.plan.step[: rd // 2]], np.float64) / 2.0 ** 64 * 2 * np.pi
    # both sides evaluate base^x in doubles: a few units of 2^-52, and 2^-62 turn of the step
    assert np.all(np.abs(got - w) <= 2.0 ** -48 * w + 2.0 ** -60)
    assert not any(plan.plan.step[rd // 2:])
    want = 0.1 * np.log(8.0) + 1 if scaling == "yarn" else 1.0
    assert abs(plan.plan.magnitude - want) <= 2.0 ** -24 * want


def test_plan_magnitude_given():
    assert kvq.RopePlan(64, scaling="yarn", factor=4.0, original_ctx=4096, magnitude=0.5).plan.magnitude == 0.5


@pytest.mark.parametrize("bad", [
    dict(head_dim=0), dict(head_dim=127), dict(head_dim=258), dict(rotary_dim=0), dict(rotary_dim=3),
    dict(rotary_dim=130), dict(interleaved=2), dict(scaling=-1), dict(scaling=5), dict(base=1.0),
    dict(base=float("nan")), dict(base=float("inf")), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("nan")),
    dict(scaling=2, rotary_dim=2), dict(scaling=2, factor=1e300, rotary_dim=4), dict(scaling=3, original_ctx=0),
    dict(scaling=3, original_ctx=4096, low=4.0, high=4.0), dict(scaling=4, original_ctx=4096, low=0.0),
    dict(scaling=4, original_ctx=4096, high=float("inf")), dict(magnitude=-1.0), dict(magnitude=float("nan")),
])
def test_plan_refusals(bad):
    st, _ = _plan(**bad)
    assert st == kvq.KVQ_ERR_INVALID
    assert b"kvq_rope_plan_init" in kvq.load_library().kvq_last_error()


def test_plan_refusals_in_python():
    lib = kvq.load_library()
    assert lib.kvq_rope_plan_init(None, None) == kvq.KVQ_ERR_INVALID
    with pytest.raises(ValueError):
        kvq.RopePlan(128, layout="both")
    with pytest.raises(ValueError):
        kvq.RopePlan(128, scaling="other")
    with pytest.raises(kvq.KvqError):
        kvq.RopePlan(128, rotary_dim=130)


@pytest.mark.parametrize("D", [64, 128])
def test_page_layout_holds_every_element_once(D):
    kb, ks, vb, vs, sp = P.tables(D)
    nibbles = np.concatenate([(2 * b + s // 4).ravel() for b, s in ((kb, ks), (vb, vs))])
    assert sorted(nibbles) == list(range(2 * PAGE_CODES(D)))
    halves = sp.ravel()
    assert sorted(halves) == list(range(PAGE_CODES(D), P.page_bytes(D), 2))
    assert kvq.paged_page_bytes(D) == P.page_bytes(D)
    rng = np.random.default_rng(0)
    f = P.unpack(P.make_pages(rng.normal(size=(3, 64, D)), rng.normal(size=(3, 64, D))), D)
    assert all(np.array_equal(f[n], P.unpack(P.pack(f, D), D)[n]) for n in f)


def PAGE_CODES(D):
    return P.PAGE * D


def test_the_format_spans_its_group():
    """Every value lies within half a step of what is held, and the values of odd slots
    count down from the maximum."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(50, 64)) * np.exp(rng.normal(size=(50, 1)) * 3)
    for down in (False, True):
        code, s, o, _ = P.quantize(x, np.full(50, down))
        held = (code.reshape(50, 2, 32) * s[..., None].astype(float) + o[..., None].astype(float)).reshape(50, 64)
        step = np.repeat(np.abs(s.astype(float)), 32, axis=1)
        far = np.repeat(np.abs(o.astype(float)), 32, axis=1)
        # half a step, and the rounding of the offset where it cuts off the group's edge
        assert np.all(np.abs(held - x) <= 0.5 * step + 2.0 ** -11 * far)
        assert np.all((s < 0) == down) and code.min() == 0 and code.max() >= 14


def test_page_bytes_refusals():
    lib = kvq.load_library()
    n = ctypes.c_size_t(0)
    assert lib.kvq_paged_page_bytes(128, None) == kvq.KVQ_ERR_INVALID
    for hd in (0, 32, 96, 256):
        assert lib.kvq_paged_page_bytes(hd, ctypes.byref(n)) == kvq.KVQ_ERR_INVALID


# ---- refusals of the C calls that come before any CUDA call ----

ADDR = 1 << 20   # an aligned address that no refused call may read


def _rope(**kw):
    _, plan = _plan(**kw.pop("plan_fields", {}))
    a = dict(plan=ctypes.addressof(plan), dtype=0, x=ADDR, xt=128, xh=128, pos=ADDR, T=4, H=2, out=ADDR, ot=128, oh=128)
    a.update(kw)
    return kvq.load_library().kvq_rope(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(plan=None), dict(dtype=2), dict(T=-1), dict(H=-1), dict(xt=-128), dict(xh=4), dict(ot=12), dict(ot=0),
    dict(oh=0), dict(plan_fields=dict(head_dim=12, rotary_dim=12)),
])
def test_rope_refusals(bad):
    assert _rope(**bad) == kvq.KVQ_ERR_INVALID
    assert b"kvq_rope" in kvq.load_library().kvq_last_error()


def test_rope_refuses_an_uninitialised_plan():
    empty = kvq.kvq_rope_plan()
    assert _rope(plan=ctypes.addressof(empty)) == kvq.KVQ_ERR_INVALID


def _append(**kw):
    _, plan = _plan(**kw.pop("plan_fields", {}))
    a = dict(plan=ctypes.addressof(plan), dtype=0, k=ADDR, kt=128, kh=128, v=ADDR, vt=128, vh=128, slots=ADDR, pos=ADDR,
             T=4, Hkv=2, hd=128, pages=ADDR, n_pages=3, q=None, qt=0, qh=0, Hq=0, q_out=None, ot=0, oh=0)
    a.update(kw)
    return kvq.load_library().kvq_paged_append(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=7), dict(hd=96), dict(T=-1), dict(Hkv=0), dict(n_pages=0), dict(n_pages=(1 << 25) + 1), dict(pos=None),
    dict(plan=None), dict(plan=None, pos=None, q=ADDR, q_out=ADDR, Hq=2), dict(q=ADDR, Hq=2), dict(q_out=ADDR, Hq=2),
    dict(q=ADDR, q_out=ADDR, Hq=0), dict(Hq=-1), dict(kt=3), dict(vh=-8),
    dict(plan_fields=dict(head_dim=64, rotary_dim=64)),
])
def test_append_refusals(bad):
    assert _append(**bad) == kvq.KVQ_ERR_INVALID
    assert b"kvq_paged_append" in kvq.load_library().kvq_last_error()


@pytest.mark.parametrize("bad", [dict(dtype=-1), dict(hd=32), dict(T=-2), dict(Hkv=0), dict(n_pages=0), dict(kt=4),
                                 dict(vt=0), dict(kh=0)])
def test_gather_refusals(bad):
    a = dict(pages=ADDR, n_pages=3, slots=ADDR, T=4, Hkv=2, hd=128, dtype=0, k=ADDR, kt=256, kh=128, v=ADDR, vt=256, vh=128)
    a.update(bad)
    assert kvq.load_library().kvq_paged_gather(*a.values(), None) == kvq.KVQ_ERR_INVALID
    assert b"kvq_paged_gather" in kvq.load_library().kvq_last_error()


def _attend(**kw):
    a = dict(dtype=0, q=ADDR, qt=1024, qh=128, pages=ADDR, n_pages=9, table=ADDR, ts=4, max_pages=4, lens=ADDR, B=2, Q=1,
             Hq=8, Hkv=2, hd=128, window=0, scale=0.0, out=ADDR, lse=None, ws=ADDR, wb=1 << 30)
    a.update(kw)
    return kvq.load_library().kvq_paged_attention(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(B=-1), dict(B=2049), dict(Q=0), dict(Q=65), dict(Hq=7), dict(Hkv=0), dict(Hq=0),
    dict(Hq=130, Hkv=2), dict(hd=256), dict(n_pages=0), dict(max_pages=0), dict(max_pages=(1 << 24) + 1), dict(max_pages=1 << 24, B=64), dict(ts=-1),
    dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(qt=-8), dict(qh=3),
])
def test_attention_refusals(bad):
    assert _attend(**bad) == kvq.KVQ_ERR_INVALID
    assert b"kvq_paged_attention" in kvq.load_library().kvq_last_error()


def test_empty_calls_do_nothing():
    assert _rope(T=0) == kvq.KVQ_OK and _rope(H=0) == kvq.KVQ_OK
    assert _append(T=0) == kvq.KVQ_OK and _attend(B=0) == kvq.KVQ_OK


def test_workspace_refusals():
    lib = kvq.load_library()
    n = ctypes.c_size_t(0)
    assert lib.kvq_paged_attention_workspace(1, 1, 8, 2, 128, None) == kvq.KVQ_ERR_INVALID
    assert lib.kvq_paged_attention_workspace(1, 1, 7, 2, 128, ctypes.byref(n)) == kvq.KVQ_ERR_INVALID


def test_python_refuses_cpu_tensors_and_odd_operands():
    plan = kvq.RopePlan(128)
    x, pos = torch.zeros(3, 2, 128, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    pages = torch.zeros(2, 2, kvq.paged_page_bytes(128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.rope(x, pos, plan)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.paged_append(pages, x, x, pos)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.paged_gather(pages, pos, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.paged_attention(x, pages, pos.reshape(3, 1), pos, x)
    with pytest.raises(ValueError):
        kvq.rope(x[0], pos, plan)
    with pytest.raises(ValueError):
        kvq.paged_attention(x[0], pages, pos.reshape(3, 1), pos, x)


@pytest.mark.parametrize("bad", [dict(xt=256), dict(xh=256), dict(ot=256), dict(oh=256)])
def test_rope_in_place_needs_the_same_strides(bad):
    assert _rope(**bad) == kvq.KVQ_ERR_INVALID
    assert b"same strides" in kvq.load_library().kvq_last_error()


def test_more_refusals_before_any_cuda_call():
    lib = kvq.load_library()
    assert _attend() == kvq.KVQ_ERR_INVALID and b"out must not be q" in lib.kvq_last_error()
    for status in (_append(Hkv=4097), _attend(Hkv=4097, Hq=4097)):
        assert status == kvq.KVQ_ERR_INVALID and b"n_kv_heads" in lib.kvq_last_error()


def test_rows_of_outputs_must_not_overlap():
    lib = kvq.load_library()
    for kw in (dict(ot=120), dict(oh=64)):
        assert _rope(x=ADDR + 4096, **kw) == kvq.KVQ_ERR_INVALID and b"must not overlap" in lib.kvq_last_error()
    a = dict(pages=ADDR, n_pages=3, slots=ADDR, T=4, Hkv=2, hd=128, dtype=0, k=ADDR, kt=256, kh=128, v=ADDR, vt=256, vh=120)
    assert lib.kvq_paged_gather(*a.values(), None) == kvq.KVQ_ERR_INVALID and b"must not overlap" in lib.kvq_last_error()

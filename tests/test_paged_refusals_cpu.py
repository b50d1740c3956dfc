"""Further refusals of the paged cache's and the rotary calls that come before any CUDA call."""

import pytest

import certified_quantized_kv_gb300 as kvq
from test_paged_cpu import ADDR, _append, _attend, _plan, _rope

FAR = ADDR + (1 << 16)


def _error():
    return kvq.load_library().kvq_last_error()


def _gather(**kw):
    a = dict(pages=ADDR, n_pages=3, slots=ADDR, T=4, Hkv=2, hd=128, dtype=0, k=ADDR, kt=256, kh=128, v=FAR, vt=256, vh=128)
    a.update(kw)
    return kvq.load_library().kvq_paged_gather(*a.values(), None)


@pytest.mark.parametrize("ts,hs,meet", [(128, 128, True), (256, 192, True), (192, 256, True), (384, 384, True), (256, 128, False),
                                        (128, 512, False), (640, 256, False), (248, 128, True), (128, 504, True)])
def test_rows_that_meet_although_each_stride_holds_one(ts, hs, meet):
    """Four tokens of two heads: token t + 1's first head on token t's second one."""
    calls = [(b"out: rows", lambda: _rope(x=FAR, xt=256, ot=ts, oh=hs)),
             (b"q_out: rows", lambda: _append(q=FAR, qt=256, qh=128, Hq=2, q_out=2 * FAR, ot=ts, oh=hs)),
             (b"k and v: rows", lambda: _gather(kt=ts, kh=hs)), (b"k and v: rows", lambda: _gather(vt=ts, vh=hs))]
    for name, call in calls:
        # (what is not refused for its rows fails for want of a device, or of device memory)
        assert call() != kvq.KVQ_OK and (name in _error()) == meet, (name, _error())


def test_the_same_buffer_for_two_outputs_or_for_an_output_and_another_input():
    assert _gather(v=ADDR) == kvq.KVQ_ERR_INVALID and b"must not overlap" in _error()
    for other in ("k", "v"):
        assert _append(**{other: FAR}, q=2 * FAR, q_out=FAR, qt=256, qh=128, ot=256, oh=128, Hq=2) == kvq.KVQ_ERR_INVALID
        assert b"q_out must not be k or v" in _error()


@pytest.mark.parametrize("scale", [2.9e38, -3.4e38])
def test_scales_whose_base_2_form_fp32_does_not_hold(scale):
    assert _attend(scale=scale, out=FAR) == kvq.KVQ_ERR_INVALID and b"scale" in _error()


@pytest.mark.parametrize("magnitude", [3.5e38, 1e300])
def test_magnitudes_that_fp32_does_not_hold(magnitude):
    assert _plan(magnitude=magnitude)[0] == kvq.KVQ_ERR_INVALID and b"magnitude" in _error()
    assert _plan(magnitude=3.4e38)[0] == kvq.KVQ_OK

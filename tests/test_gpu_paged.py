"""The paged 4-bit cache on the GPU: rotary positions, the append that rotates and
quantises, the read-back and attention over the pages, each against its definition in 64
bits (tests/_paged.py), and all of them together as a serving loop uses them.

Tolerances, for an element type of half step eps/2 (binary16 2^-11, bfloat16 2^-8, relative
to the value) with a smallest step TINY:
  rotation     |y| eps/2 + TINY for the one rounding, plus (|a| + |b|) m 2^-21 for fp32: the angle is
               right to 2^-32 half turns and rounded to fp32 (2^-25 half turns, 2^-23.3 rad), the
               sine and cosine functions are within 2 units (2^-23), products and sum 3 2^-24:
               2^-23.3 + 2^-23 + 3 2^-24 < 2^-21.4
  held values  a code may differ from the oracle's only where the quotient lies within 2^-16 of
               a half (fp32: (x - o) / s <= 15.5 with relative error 3 2^-24, and the rotated key's
               own error, 2^-21 of its pair, over a step that is 1/15 of the group's range or more)
  attention    |out| eps/2 + TINY for the rounding; scores are sums of 128 exact products in
               fp32 with truncating adders: within 2^-17 of scale sum |q| (s code + |o|), called A
               below (MMA accumulation was measured within 2^-18.5 of the sum of magnitudes),
               plus 2^-22 of their own size for the exponent; weights and sums 2^-18:
               (2 (2^-17 A) + 2^-17) sum p |v^|, and |o| + s code <= 3 max |k^| of a group bounds A
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
TYPES = [torch.float16, torch.bfloat16]
ROPES = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=4.0),
         dict(base=500000.0, scaling="parts", factor=8.0, original_ctx=8192, high=4.0),
         dict(scaling="yarn", factor=16.0, original_ctx=4096)]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _randn(shape, dt, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * scale).to(dt).cuda()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------------------

def _check_rope(got, x, pos, plan_kw, D, rd, inter):
    w = P.frequencies(rd, **plan_kw)
    m = 0.1 * np.log(plan_kw["factor"]) + 1 if plan_kw.get("scaling") == "yarn" else 1.0
    xf = _f64(x)
    ref = P.rope(xf, pos.cpu().numpy(), rd, inter, w, m)
    ab = P.rope(np.abs(xf), np.zeros(len(pos)), rd, inter, w, 1.0)   # |x|, pairs in place
    i0, i1 = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, rd // 2), slice(rd // 2, rd))
    both = np.zeros_like(xf)
    both[..., i0] = both[..., i1] = ab[..., i0] + ab[..., i1]
    tol = np.abs(ref) * HALF[x.dtype] + TINY[x.dtype] + both * m * 2.0 ** -21 * (1 + HALF[x.dtype])
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= tol), float((err - tol).max())
    assert torch.equal(got[..., rd:], x[..., rd:])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rd,kind", [(1, 1, 128, 128, 0), (5, 40, 128, 128, 3), (67, 3, 64, 64, 1), (9, 2, 8, 2, 0),
                                           (33, 5, 128, 26, 2), (130, 7, 96, 96, 4), (3, 1, 256, 256, 3),
                                           (301, 9, 80, 32, 4), (17, 13, 128, 120, 1), (2, 33, 256, 64, 2),
                                           (1000, 1, 64, 48, 0), (70, 2, 136, 112, 1)])
def test_rope(T, H, D, rd, kind, layout, dt):
    kw = ROPES[kind]
    if kw.get("scaling") == "ntk" and rd < 4:
        kw = {}
    plan = kvq.RopePlan(D, rotary_dim=rd, layout=layout, **kw)
    x = _randn((T, H, D), dt, T + D)
    pos = torch.randint(-2000000, 2000000, (T,), generator=_gen(rd)).int().cuda()
    out = kvq.rope(x, pos, plan)
    _check_rope(out, x, pos, kw, D, rd, layout == "interleaved")
    same = x.clone()
    assert kvq.rope(same, pos, plan, out=same) is same and torch.equal(same, out)   # in place


def test_rope_extreme_positions():
    plan = kvq.RopePlan(128, base=500000.0)
    pos = _ints([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 123456789])
    x = _randn((7, 2, 128), torch.float16, 3)
    out = kvq.rope(x, pos, plan)
    assert torch.equal(out[0], x[0])
    # the double frequencies of both sides agree to 2^-48 relative: 2^31 positions turn that into
    # 2^-17 rad beside the tolerance above
    ref = P.rope(_f64(x), pos.cpu().numpy(), 128, False, P.frequencies(128, base=500000.0))
    assert np.abs(_f64(out) - ref).max() <= 8 * (2.0 ** -11 + 2.0 ** -16)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H,D,rd", [(7, 40, 128, 42), (3, 13, 256, 250), (500, 33, 64, 18), (40, 9, 80, 74), (2, 70, 128, 4),
                                      (5000, 3, 128, 52), (1, 1, 16, 10)])
def test_rope_of_halves_across_vectors(T, H, D, rd, dt):
    """Halves that are no multiple of 4: out of place into a wider buffer, and in place."""
    kw = ROPES[3]
    plan = kvq.RopePlan(D, rotary_dim=rd, **kw)
    x = _randn((T, H, D), dt, T + H)
    pos = torch.randint(-100000, 100000, (T,), generator=_gen(rd)).int().cuda()
    wide = torch.full((T, H + 1, D), 3.0, dtype=dt, device="cuda")
    out = kvq.rope(x, pos, plan, out=wide[:, :H])
    _check_rope(out, x, pos, kw, D, rd, False)
    assert (wide[:, H] == 3).all()
    same = x.clone()
    kvq.rope(same, pos, plan, out=same)
    assert torch.equal(same, out)
    if D in (64, 128):      # the same rotation beside the append
        pages = torch.zeros(-(-T // 64), H, kvq.paged_page_bytes(D), dtype=torch.uint8, device="cuda")
        q = x.clone()
        kvq.paged_append(pages, x, x, torch.arange(T).int().cuda(), positions=pos, plan=plan, q=x, q_out=q)
        assert torch.equal(q, out)


def test_rope_phases_where_the_products_cancel():
    """a cos - b sin with a / b close to tan: what is left shows the cosine's and the sine's own
    errors.  Both lie within 2^-23.5 (series, roundings and the angle's), the two products and
    their sum round by 3 2^-24 of 32768: 32768 (sqrt 2 2^-23.5 + 3 2^-24), beside the one
    rounding to the element type and, for the frequencies in double, |p| 2^-50 turns."""
    T, plan = 6000, kvq.RopePlan(128, base=500000.0)
    pos = torch.randint(-2 ** 27, 2 ** 27, (T,), generator=_gen(3)).int()
    pos[:9] = torch.tensor([0, 1, -1, 2, 3, -2 ** 31, 2 ** 31 - 1, 5, 7]).int()
    ang = pos.numpy().astype(np.float64)[:, None] * P.frequencies(128, base=500000.0)
    x = np.concatenate([32768 * np.sin(ang), 32768 * np.cos(ang)], 1)[:, None]
    x = torch.from_numpy(x).half().cuda()
    out = _f64(kvq.rope(x, pos.cuda(), plan))
    ref = P.rope(_f64(x), pos.numpy(), 128, False, P.frequencies(128, base=500000.0))
    far = np.abs(pos.numpy().astype(np.float64))[:, None, None] * 2.0 ** -50 * 2 * np.pi * 65536
    tol = np.abs(ref) * 2.0 ** -11 + 2.0 ** -24 + 32768 * (2 ** 0.5 * 2.0 ** -23.5 + 3 * 2.0 ** -24) + far
    assert np.all(np.abs(out - ref) <= tol), float((np.abs(out - ref) - tol).max())
    assert np.abs(ref[..., :64]).max() < 40      # it does cancel


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [128, 36])
def test_rope_strided_views(layout, rd):
    """q and k slices of one fused projection, in and out of place; what lies between the
    rows stays as it was."""
    T, D = 19, 128
    plan = kvq.RopePlan(D, rotary_dim=rd, layout=layout)
    fused = _randn((T, 4 + 2 + 2, D), torch.bfloat16, 9)
    pos = torch.arange(T).int().cuda() * 31
    q, k = fused[:, :4], fused[:, 4:6]
    want_q, want_k = kvq.rope(q.contiguous(), pos, plan), kvq.rope(k.contiguous(), pos, plan)
    keep = fused.clone()
    big = torch.full((T, 9, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    view = big[:, 1:9:2, :D]
    assert torch.equal(kvq.rope(q, pos, plan, out=view), want_q) and torch.equal(view, want_q)
    assert (big[:, 0::2] == 7).all() and (big[..., D:] == 7).all()
    kvq.rope(fused[:, :6], pos, plan, out=fused[:, :6])
    assert torch.equal(fused[:, :4], want_q) and torch.equal(fused[:, 4:6], want_k)
    assert torch.equal(fused[:, 6:], keep[:, 6:])
    # one row broadcast over the heads
    one = _randn((T, 1, D), torch.bfloat16, 5)
    assert torch.equal(kvq.rope(one.expand(T, 3, D), pos, plan), kvq.rope(one.expand(T, 3, D).contiguous(), pos, plan))


def test_rope_transpose_is_the_gradient():
    """<R(p) x, y> = <x, R(-p) y> for every x and y, and the difference quotient of the
    (linear) call along y."""
    T, H, D = 11, 3, 128
    for kw in (dict(), dict(scaling="yarn", factor=8.0, original_ctx=4096, layout="interleaved", rotary_dim=96)):
        plan = kvq.RopePlan(D, **kw)
        x, y = _randn((T, H, D), torch.float16, 1), _randn((T, H, D), torch.float16, 2)
        pos = torch.arange(T).int().cuda() * 1001
        fx, ty = kvq.rope(x, pos, plan), kvq.rope(y, -pos, plan)
        a, b = (_f64(fx) * _f64(y)).sum(-1), (_f64(x) * _f64(ty)).sum(-1)
        m = plan.plan.magnitude
        # two roundings of 2^-11 each per element, against sum |x_i| |y_i| pairs
        tol = 2 * 2.0 ** -11 * m * (np.abs(_f64(x)).sum(-1) * np.abs(_f64(y)).max(-1)) + 2.0 ** -10
        assert np.all(np.abs(a - b) <= tol)
        quot = (_f64(kvq.rope((x.float() + y.float()).half(), pos, plan)) - _f64(fx))
        want = _f64(kvq.rope(y, pos, plan))
        scale = np.abs(_f64(x)).max() + np.abs(_f64(y)).max()
        assert np.abs(quot - want).max() <= 4 * 2.0 ** -11 * 2 * m * scale


def test_rope_refusals():
    plan = kvq.RopePlan(128)
    x, pos = torch.zeros(4, 2, 128, dtype=torch.float16, device="cuda"), _ints([0, 1, 2, 3])
    for args in ((x.float(), pos), (x, pos.long()), (x, pos[:3]), (x[..., :64], pos), (x.cpu(), pos), (x, pos.cpu()),
                 (x.transpose(1, 2), pos)):
        with pytest.raises(ValueError):
            kvq.rope(*args, plan)
    with pytest.raises(ValueError):
        kvq.rope(x, pos, plan, out=x.bfloat16())
    lib = kvq.load_library()

    def call(xp, out, pp=pos.data_ptr(), st=256):
        return lib.kvq_rope(plan.address, 0, xp, st, 128, pp, 4, 2, out, 256, 128, None)

    host = torch.zeros(4, 2, 128, dtype=torch.float16)
    assert call(host.data_ptr(), x.data_ptr()) == kvq.KVQ_ERR_INVALID
    assert call(x.data_ptr() + 2, x.data_ptr()) == kvq.KVQ_ERR_INVALID
    assert call(x.data_ptr(), None) == kvq.KVQ_ERR_INVALID
    assert call(x.data_ptr(), x.data_ptr(), None) == kvq.KVQ_ERR_INVALID
    assert call(x.data_ptr(), x.data_ptr(), st=252) == kvq.KVQ_ERR_INVALID
    torch.cuda.synchronize()


# --------------------------------------------------------------------------------------
# append and read-back
# --------------------------------------------------------------------------------------

def _append_case(T, Hkv, D, dt, seed, n_pages=None, kscale=1.0, vscale=1.0, pad=True):
    n_pages = n_pages or -(-T // 64) + 2
    k, v = _randn((T, Hkv, D), dt, seed, kscale), _randn((T, Hkv, D), dt, seed + 1, vscale)
    slots = torch.randperm(n_pages * 64, generator=_gen(seed + 2))[:T].int()
    if pad:
        slots[3::7] = -1
        slots[5::19] = n_pages * 64 + 5
    pos = torch.randint(0, 200000, (T,), generator=_gen(seed + 3)).int()
    pages = torch.randint(0, 256, (n_pages, Hkv, P.page_bytes(D)), generator=_gen(seed + 4)).to(torch.uint8)
    return k, v, slots.cuda(), pos.cuda(), pages.cuda()


def _check_append(before, after, k, v, slots, D, near=2.0 ** -16, key_err=None):
    """The given slots hold the oracle's quantisation of k and v (float64), every other byte
    is as before."""
    n_pages, Hkv = before.shape[:2]
    f0, f1 = P.unpack(before.cpu().numpy(), D), P.unpack(after.cpu().numpy(), D)
    slots = slots.cpu().numpy()
    ok = (slots >= 0) & (slots < n_pages * 64)
    page, at = slots[ok] // 64, slots[ok] % 64
    touched = np.zeros((n_pages, 64), bool)
    touched[page, at] = True
    for n in f0:
        a, b = (f[n].view(np.uint16) if f[n].dtype == np.float16 else f[n] for f in (f0, f1))
        keep = np.broadcast_to(~touched[:, None, :, None], a.shape)
        assert np.array_equal(a[keep], b[keep]), n
    for x, down, c, s, o in ((k, np.zeros(ok.sum(), bool), "kc", "ks", "ko"), (v, at % 2 == 1, "vc", "vs", "vo")):
        code, sc, of, quot = P.quantize(x[ok], np.broadcast_to(down[:, None], (ok.sum(), Hkv)))
        got_s, got_o = f1[s][page, :, at].astype(float), f1[o][page, :, at].astype(float)
        got = f1[c][page, :, at]
        if c == "vc" or key_err is None:   # no rotation: scale and offset are exact
            assert np.array_equal(got_s, sc.astype(float)) and np.array_equal(got_o, of.astype(float))
            margin = near
        else:      # a rotated key within key_err of the exact one: one binary16 step of o and s
            assert np.all(np.abs(got_o - of) <= 2.0 ** -10 * np.abs(of) + 2.0 ** -24)
            assert np.all(np.abs(got_s - sc) <= 2.0 ** -10 * np.abs(sc) + 2.0 ** -24 + 2.0 ** -13 * np.abs(of))
            # the held value is within half a step of the exact key and what the fp32 rotation,
            # the offset's rounding and the scale's change move
            sx = np.repeat(np.abs(got_s), 32, -1)
            held = got * np.repeat(got_s, 32, -1) + np.repeat(got_o, 32, -1)
            err = np.abs(held - np.clip(x[ok], -65504, 65504))
            assert np.all(err <= 0.5 * sx * (1 + 2.0 ** -14) + 2.0 ** -11 * np.repeat(np.abs(got_o), 32, -1) + 16 * key_err)
            margin = None
        if margin is None:
            # codes: equal but where the quotient is near a half, or the scale moved
            moved = np.repeat((got_s != sc) | (got_o != of), 32, -1)
            frac = np.abs(quot - np.floor(quot) - 0.5)
            slack = 4 * key_err / np.maximum(sx, 2.0 ** -24) + near
            assert np.all((got == code) | moved | (frac <= slack))
            assert moved.mean() <= 0.02
        else:
            frac = np.abs(quot - np.floor(quot) - 0.5)
            assert np.all((got == code) | (frac <= margin))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,Hkv,D", [(1, 1, 128), (3, 2, 64), (64, 8, 128), (131, 3, 128), (300, 5, 64), (1029, 1, 128)])
def test_append_without_rotation(T, Hkv, D, dt):
    k, v, slots, _, pages = _append_case(T, Hkv, D, dt, seed=T + D)
    before = pages.clone()
    kvq.paged_append(pages, k, v, slots)
    _check_append(before, pages, _f64(k), _f64(v), slots, D)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,Hq,Hkv,D,rd,layout,kind", [
    (1, 4, 1, 128, 128, "half", 0), (64, 32, 8, 128, 128, "half", 3), (77, 6, 3, 64, 64, "interleaved", 4),
    (130, 0, 2, 128, 26, "half", 1), (41, 5, 5, 128, 120, "interleaved", 2), (200, 16, 1, 64, 48, "half", 0),
    (33, 7, 7, 64, 18, "interleaved", 0), (2100, 2, 2, 128, 64, "half", 0)])
def test_append_with_rotation(T, Hq, Hkv, D, rd, layout, kind, dt):
    kw = ROPES[kind]
    plan = kvq.RopePlan(D, rotary_dim=rd, layout=layout, **kw)
    k, v, slots, pos, pages = _append_case(T, Hkv, D, dt, seed=T + rd)
    before = pages.clone()
    q = _randn((T, Hq, D), dt, 77) if Hq else None
    q_out = torch.empty_like(q) if Hq else None
    kvq.paged_append(pages, k, v, slots, positions=pos, plan=plan, q=q, q_out=q_out)
    w = P.frequencies(rd, **kw)
    m = plan.plan.magnitude
    rk = P.rope(_f64(k), pos.cpu().numpy(), rd, layout == "interleaved", w, m)
    _check_append(before, pages, rk, _f64(v), slots, D, key_err=2 * m * 2.0 ** -21 * float(k.abs().max()))
    if Hq:
        _check_rope(q_out, q, pos, kw, D, rd, layout == "interleaved")
        again = pages.clone()
        kvq.paged_append(again, k, v, slots, positions=pos, plan=plan, q=q, q_out=q)     # in place
        assert torch.equal(q, q_out) and torch.equal(again, pages)


@pytest.mark.parametrize("D", [64, 128])
def test_append_edges(D):
    """Constant groups, groups spanning the whole binary16 range, elements beyond it, tiny
    values, exact ties, and positions of padding tokens (rotated q only)."""
    T, H = 40, 2
    k = torch.zeros(T, H, D)
    v = torch.zeros(T, H, D)
    k[0], v[0] = 3.25, -1.5                                   # constant: scale 0
    k[1], v[1] = 1e-7, 2e-7                                   # subnormal range
    k[2, :, ::2], v[2, :, ::2] = 65504.0, -65504.0            # the largest scale
    k[3, :, 1::2], v[3, :, 1::2] = -65504.0, 65504.0
    j = torch.arange(D) % 32
    k[4:20] = torch.where(j == 31, 15.0, torch.where(j == 0, 0.0, j / 2.0 + 0.0))   # ties at halves
    v[4:20] = k[4:20]
    k[20:] = torch.randn(20, H, D, generator=_gen(1)) * 1e3
    v[20:] = torch.randn(20, H, D, generator=_gen(2)) * 1e-3
    pages = torch.zeros(2, H, P.page_bytes(D), dtype=torch.uint8, device="cuda")
    slots = _ints(list(range(30, 30 + T)))
    for dt in TYPES:
        kd, vd = k.to(dt).cuda(), v.to(dt).cuda()
        if dt == torch.bfloat16:
            kd[20, 0, 3], vd[21, 0, 5] = 1e30, -1e30          # held as +-65504
        before = pages.clone()
        kvq.paged_append(pages, kd, vd, slots)
        _check_append(before, pages, _f64(kd), _f64(vd), slots, D)


def test_append_strided_and_one_token():
    T, Hkv, D = 21, 2, 128
    fused = _randn((T, 4 + 2 * Hkv, D), torch.float16, 4)
    plan = kvq.RopePlan(D)
    slots, pos = _ints(list(range(64 + 5, 64 + 5 + T))), _ints(list(range(100, 100 + T)))
    a = torch.zeros(3, Hkv, P.page_bytes(D), dtype=torch.uint8, device="cuda")
    b, c = a.clone(), a.clone()
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    qa = torch.empty(T, 4, D, dtype=torch.float16, device="cuda")
    kvq.paged_append(a, k, v, slots, positions=pos, plan=plan, q=q, q_out=qa)
    kvq.paged_append(b, k.contiguous(), v.contiguous(), slots, positions=pos, plan=plan)
    for t in range(T):      # one token at a time, as a decoding step does
        kvq.paged_append(c, k[t:t + 1], v[t:t + 1], slots[t:t + 1], positions=pos[t:t + 1], plan=plan)
    assert torch.equal(a, b) and torch.equal(a, c)
    assert torch.equal(qa, kvq.rope(q, pos, plan))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,Hkv,D", [(1, 1, 64), (70, 3, 128), (333, 4, 64), (64, 8, 128)])
def test_gather(T, Hkv, D, dt):
    """Bit for bit o + s code in fp32, rounded once; zeros for slots outside the pool."""
    n_pages = 5 + T // 64
    g = np.random.default_rng(T)
    pages = P.make_pages(g.normal(size=(n_pages * Hkv, 64, D)) * 3, g.normal(size=(n_pages * Hkv, 64, D)))
    slots = torch.randint(0, n_pages * 64, (T,), generator=_gen(T)).int()
    slots[2::5] = -7
    slots[4::11] = n_pages * 64
    k = torch.full((T, Hkv, D), 9.0, dtype=dt, device="cuda")
    big = torch.full((T, Hkv, 2 * D), 9.0, dtype=dt, device="cuda")
    v = big[..., :D]
    kvq.paged_gather(torch.from_numpy(pages).reshape(n_pages, Hkv, -1).cuda(), slots.cuda(), k, v)
    kf, vf = (x.reshape(n_pages, Hkv, 64, D) for x in P.values(P.unpack(pages, D), D, np.float32))
    s = slots.numpy()
    ok = (s >= 0) & (s < n_pages * 64)
    sc = np.where(ok, s, 0)
    for got, want in ((k, kf), (v, vf)):
        want = np.where(ok[:, None, None], want[sc // 64, :, sc % 64], np.float32(0))
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dt))
    assert (big[..., D:] == 9).all()


def test_append_and_gather_refusals():
    T, H, D = 4, 2, 128
    k, slots, pos = torch.zeros(T, H, D, dtype=torch.float16, device="cuda"), _ints([0, 1, 2, 3]), _ints([0, 1, 2, 3])
    pages = torch.zeros(2, H, 10240, dtype=torch.uint8, device="cuda")
    plan, p64 = kvq.RopePlan(D), kvq.RopePlan(64)
    bad = [dict(v=k.bfloat16()), dict(v=k[:3]), dict(slots=slots.long()), dict(pages=pages[:, :1]),
           dict(pages=pages[..., :5120]), dict(pages=pages.cpu()), dict(plan=plan), dict(positions=pos),
           dict(plan=plan, positions=pos, q=k), dict(plan=plan, positions=pos, q=k, q_out=k.bfloat16()),
           dict(q=k, q_out=k), dict(plan=p64, positions=pos), dict(k=k.transpose(0, 2)), dict(k=k[..., :96], v=k[..., :96])]
    for kw in bad:
        args = dict(pages=pages, k=k, v=k, slots=slots)
        args.update(kw)
        with pytest.raises((ValueError, kvq.KvqError)):
            kvq.paged_append(**args)
    for kw in (dict(v=k[:2]), dict(k=k.float(), v=k.float()), dict(slots=slots[:1]), dict(pages=pages.float())):
        args = dict(pages=pages, slots=slots, k=k.clone(), v=k.clone())
        args.update(kw)
        with pytest.raises((ValueError, kvq.KvqError)):
            kvq.paged_gather(**args)
    with pytest.raises(ValueError):      # the pool is for head_dim 128
        kvq.paged_append(pages, k[..., :64], k[..., :64], slots)
    with pytest.raises(kvq.KvqError):    # k is not 16-byte aligned
        kvq.paged_append(torch.zeros(2, H, 5120, dtype=torch.uint8, device="cuda"), k[..., 1:65], k[..., :64], slots)
    assert not pages.any()


# --------------------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------------------

def _cache(lens, Hkv, D, seed, kscale=1.0, vscale=1.0, spare=3, stale="nan"):
    """Pages holding len tokens per sequence in shuffled order; what lies behind a
    sequence's last token, and the unused pages, is NaN scales and offsets over random codes."""
    g = np.random.default_rng(seed)
    need = [-(-max(n, 0) // 64) for n in lens]
    n_pages = sum(need) + spare
    pages = P.make_pages(g.normal(size=(n_pages * Hkv, 64, D)) * kscale, g.normal(size=(n_pages * Hkv, 64, D)) * vscale)
    pages = pages.reshape(n_pages, Hkv, -1)
    order = g.permutation(n_pages)
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    used = np.zeros((n_pages, 64), bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, : need[b]] = order[at: at + need[b]]
        for j in range(need[b]):
            used[table[b, j], : min(64, n - 64 * j)] = True
        at += need[b]
    f = P.unpack(pages, D)
    if stale == "nan":
        for name in ("ks", "ko", "vs", "vo"):
            f[name][np.broadcast_to(~used[:, None, :, None], f[name].shape)] = np.float16(np.nan)
    kv = P.values(f, D)
    return P.pack(f, D), table, kv


def _tokens(kv, table, b, h, n):
    k = kv[0][table[b, : -(-n // 64)], h].reshape(-1, kv[0].shape[-1])[:n]
    v = kv[1][table[b, : -(-n // 64)], h].reshape(-1, kv[1].shape[-1])[:n]
    return k, v


def _check_attention(out, lse, q, kv, table, lens, window, scale, heads=None):
    B, Q, Hq, D = q.shape
    Hkv = kv[0].shape[1]
    n = Hq // Hkv
    qf, of, lf, dt = _f64(q), _f64(out).reshape(q.shape), _f64(lse).reshape(q.shape[:3]), q.dtype
    scale = scale or 1 / np.sqrt(D)
    for b in range(B):
        L = max(0, int(lens[b]))
        ends = [max(0, L - Q + 1 + i) for i in range(Q)]
        for h in heads or range(Hkv):
            r = slice(h * n, (h + 1) * n)
            k, v = _tokens(kv, table, b, h, L)
            ref, rl, pv, qk = P.attention(qf[b][:, r], k, v, ends, window, scale)
            dS = 3 * qk * 2.0 ** -17 + np.where(np.isfinite(rl), np.abs(rl), 0) * 2.0 ** -22 + 2.0 ** -18
            err = np.abs(of[b][:, r] - ref)
            vmax = np.abs(v).max() if L else 0.0
            tol = np.abs(ref) * HALF[dt] + TINY[dt] + (2 * dS[..., None] + 2.0 ** -17) * pv + 2.0 ** -30 * vmax
            assert np.all(err <= tol), (b, h, float((err - tol).max()), float(err.max()))
            seen = np.isfinite(rl)
            assert np.array_equal(seen, np.isfinite(lf[b][:, r])), (b, h)
            assert np.all(lf[b][:, r][~seen] == -np.inf) and np.all(of[b][:, r][~seen] == 0)
            assert np.all(np.abs(lf[b][:, r] - rl)[seen] <= (dS + np.abs(rl) * 2.0 ** -22)[seen]), (b, h)


def _attend(q, pages, table, lens, window=0, scale=None, **kw):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:-1], float("nan"), device="cuda")
    ws = kvq.paged_attention(q, pages, table, lens, out, lse=lse, scale=scale, window=window, **kw)
    return out, lse, ws


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,window", [
    ([1], 1, 1, 1, 128, 0),
    ([64], 1, 4, 1, 128, 0),
    ([63, 65, 0, 128], 1, 32, 8, 128, 0),
    ([200, 1, 0, 777, 64], 1, 6, 2, 128, 0),             # three query heads to a KV head
    ([1000], 1, 8, 8, 128, 0),                           # one
    ([500, 37], 1, 14, 2, 128, 0),                       # seven
    ([130, 321], 1, 8, 1, 64, 0),
    ([90, 64, 3], 1, 24, 3, 64, 100),
    ([300, 5], 1, 16, 1, 128, 0),
    ([450], 1, 48, 2, 64, 0),                            # 24
    ([129], 1, 64, 1, 128, 0),                           # 64
    ([300, 2, 0, 65], 4, 8, 2, 128, 0),                  # drafted tokens, some before the first one
    ([1, 700], 8, 10, 5, 128, 0),
    ([400, 66], 5, 6, 2, 64, 70),
    ([200, 63], 16, 4, 1, 128, 0),                       # 64 rows
    ([513], 3, 1, 1, 128, 1),                            # every query sees its own token only
    ([640, 64], 2, 12, 1, 128, 64),
    ([100], 64, 2, 2, 64, 33),
    ([-5, 70], 1, 4, 2, 128, 0),                         # a negative length counts as empty
])
def test_attention(lens, Q, Hq, Hkv, D, window, dt):
    pages, table, kv = _cache(lens, Hkv, D, seed=sum(lens) + Q)
    q = _randn((len(lens), Q, Hq, D), dt, 5, 2.0)
    out, lse, ws = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens), window)
    _check_attention(out, lse, q, kv, table, lens, window, None)
    # the same bits again, with the used workspace, and without lse
    out2, lse2, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens), window, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    out3 = torch.empty_like(out)
    kvq.paged_attention(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens), out3, window=window)
    assert torch.equal(out, out3)


def _widened(table, columns=9000):
    """The table with room for more pages: as many as make the call use its tiles of 16 rows."""
    return np.concatenate([table, np.full((len(table), columns - table.shape[1]), -1, np.int32)], 1)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,window", [
    ([300, 5], 1, 16, 1, 128, 0),
    ([450], 1, 96, 2, 64, 0),                            # 48 rows
    ([129], 1, 64, 1, 128, 0),
    ([300, 2, 0, 65], 3, 8, 2, 128, 0),                  # twelve rows
    ([1, 700], 5, 10, 5, 128, 0),                        # ten
    ([400, 66], 5, 6, 2, 64, 70),
    ([200, 63], 16, 4, 1, 128, 0),
    ([640, 64], 1, 27, 3, 128, 64),                      # nine
    ([100], 64, 2, 2, 64, 33),
    ([3000, 64 * 20], 4, 32, 8, 128, 0),                 # split over the GPU
    ([9000], 3, 32, 2, 64, 0),
    ([129] * 40 + [0] * 7, 7, 8, 4, 128, 0),
])
def test_attention_in_tiles_of_16_rows(lens, Q, Hq, Hkv, D, window, dt):
    pages, table, kv = _cache(lens, Hkv, D, seed=sum(lens) + Q)
    q = _randn((len(lens), Q, Hq, D), dt, 5, 2.0)
    wide = torch.from_numpy(_widened(table)).cuda()
    out, lse, ws = _attend(q, torch.from_numpy(pages).cuda(), wide, _ints(lens), window)
    _check_attention(out, lse, q, kv, table, lens, window, None)
    out2, lse2, _ = _attend(q, torch.from_numpy(pages).cuda(), wide, _ints(lens), window, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # tiles of 8 rows in the same workspace, then tiles of 16 again
    out3, lse3, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens), window, workspace=ws)
    _check_attention(out3, lse3, q, kv, table, lens, window, None)
    out4, lse4, _ = _attend(q, torch.from_numpy(pages).cuda(), wide, _ints(lens), window, workspace=ws)
    assert torch.equal(out, out4) and torch.equal(lse, lse4)


@pytest.mark.parametrize("lens,Hq,Hkv,D,Q", [
    ([4096 + 37], 32, 8, 128, 1),          # one sequence split over the GPU
    ([40000], 4, 1, 128, 1),               # one group split over every warp
    ([30000, 11, 0, 5000], 8, 2, 64, 1),
    ([7] * 300, 8, 2, 128, 1),             # many short sequences: several groups to a warp
    ([129] * 90 + [0] * 7, 16, 4, 128, 1),
    ([3000, 64 * 20], 32, 8, 128, 4),
    ([9000], 32, 2, 64, 3),
])
def test_attention_split_over_the_gpu(lens, Hq, Hkv, D, Q):
    pages, table, kv = _cache(lens, Hkv, D, seed=len(lens))
    q = _randn((len(lens), Q, Hq, D), torch.float16, 6)
    out, lse, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens))
    _check_attention(out, lse, q, kv, table, lens, 0, None)


def test_attention_full_layer_128k():
    """A 131072-token layer of the Llama-3.1-8B shape, one KV head's rows compared."""
    lens = [131072]
    pages, table, kv = _cache(lens, 8, 128, seed=2, spare=0)
    q = _randn((1, 1, 32, 128), torch.float16, 6)
    out, lse, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens))
    _check_attention(out, lse, q, kv, table, lens, 0, None, heads=[0, 5])


@pytest.mark.parametrize("kscale,vscale", [(30.0, 1.0), (1.0, 300.0), (1.0, 1e-3), (100.0, 8000.0), (1e-3, 1.0)])
def test_attention_scales(kscale, vscale):
    """Peaked softmax, value scales far above and below one, and scales that change by orders of
    magnitude from page to page."""
    lens = [1500, 190]
    pages, table, kv = _cache(lens, 2, 128, seed=8, kscale=kscale, vscale=vscale)
    q = _randn((2, 1, 8, 128), torch.float16, 7)
    args = torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens)
    out, lse, _ = _attend(q, *args)
    _check_attention(out, lse, q, kv, table, lens, 0, None)
    g = np.random.default_rng(3)
    n = pages.shape[0] * 2
    mixed = P.make_pages(g.normal(size=(n, 64, 128)), g.normal(size=(n, 64, 128)) * np.exp(g.normal(size=(n, 1, 1)) * 4).clip(1e-3, 1e4))
    mixed = mixed.reshape(pages.shape)
    out, lse, _ = _attend(q, torch.from_numpy(mixed).cuda(), *args[1:])
    _check_attention(out, lse, q, P.values(P.unpack(mixed, 128), 128), table, lens, 0, None)


def test_attention_small_weights_add_up():
    """One strong token before very many weak ones: weights far below the strong one's
    binary16 range still count."""
    n = 64 * 600
    g = np.random.default_rng(4)
    k = g.normal(size=(n, 128)) * 1e-3
    k[100] = 1.0
    v = np.ones((n, 128)) + g.normal(size=(n, 128)) * 0.01
    v[100] = -1.0
    pages = P.make_pages(k.reshape(-1, 64, 128), v.reshape(-1, 64, 128)).reshape(-1, 1, 10240)
    table = np.arange(600, dtype=np.int32)[None]
    kv = P.values(P.unpack(pages, 128), 128)
    q = torch.full((1, 1, 2, 128), 1.0, dtype=torch.float16, device="cuda")
    for scale in (0.05, 0.085, 0.12):     # exp(6.4), exp(10.9), exp(15.4) times the weak tokens' weight
        out, lse, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints([n]), scale=scale)
        _check_attention(out, lse, q, kv, table, [n], 0, scale)


def test_attention_operands():
    """q as a slice of a fused buffer, three-dimensional q, a wide page table, pages shared by
    sequences, a given scale, zero queries."""
    lens = [210, 150, 64]
    pages, table, kv = _cache(lens, 2, 128, seed=3)
    table[1, :2] = table[0, :2]      # a shared prefix
    dev = torch.from_numpy(pages).cuda()
    wide = torch.full((3, 40), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + table.shape[1]] = torch.from_numpy(table).cuda()
    tab = wide[:, 5:5 + table.shape[1]]
    fused = _randn((3, 8 + 4, 128), torch.bfloat16, 2)
    q = fused[:, :8]
    for scale in (None, 0.31):
        out, lse, _ = _attend(q, dev, tab, _ints(lens), scale=scale)
        _check_attention(out, lse, q[:, None], kv, table, lens, 0, scale)
    z = torch.zeros(3, 8, 128, dtype=torch.float16, device="cuda")
    out, lse, _ = _attend(z, dev, tab, _ints(lens))
    _check_attention(out, lse, z[:, None], kv, table, lens, 0, None)
    big = (fused[:, :8].float() * 1e4).half()       # scores in the hundreds of thousands
    out, lse, _ = _attend(big, dev, tab, _ints(lens))
    _check_attention(out, lse, big[:, None], kv, table, lens, 0, None)


def test_attention_entries_outside_the_pool():
    """Tokens of page-table entries outside the pool are not seen; lengths beyond the table
    are clamped to it."""
    lens = [320, 64, 100]
    pages, table, kv = _cache(lens, 1, 128, seed=5)
    table = table[:, :5].copy()
    k, v = _tokens(kv, table, 0, 0, 320)
    table[0, 1], table[0, 3], table[1, 0] = -1, pages.shape[0], -2 ** 31
    q = _randn((3, 1, 4, 128), torch.float16, 1)
    out, lse, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints([100000, 64, 100]))
    keep = np.r_[0:64, 128:192, 256:320]
    ref, rl, pv, qk = P.attention(_f64(q)[0], k[keep], v[keep], [len(keep)], 0, 1 / np.sqrt(128))
    assert np.all(np.abs(_f64(out)[0] - ref) <= np.abs(ref) * 2.0 ** -11 + 2.0 ** -24 + (6 * qk[..., None] * 2.0 ** -17 + 2.0 ** -16) * pv)
    assert np.all(_f64(out)[1] == 0) and np.all(_f64(lse)[1] == -np.inf)
    assert np.isfinite(_f64(out)[2]).all()


def test_attention_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes: the pages of its far end."""
    Hkv, D, n_pages = 8, 128, 56000
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of device memory")
    pool = torch.empty(n_pages, Hkv, 10240, dtype=torch.uint8, device="cuda")
    ids = [n_pages - 1, n_pages - 5, 2, n_pages - 3]
    k, v = _randn((250, Hkv, D), torch.float16, 1), _randn((250, Hkv, D), torch.float16, 2)
    slots = _ints([ids[t // 64] * 64 + t % 64 for t in range(250)])
    kvq.paged_append(pool, k, v, slots)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    kvq.paged_gather(pool, slots, kb, vb)
    small = torch.zeros(4, Hkv, 10240, dtype=torch.uint8, device="cuda")
    near = torch.arange(250).int().cuda()
    kvq.paged_append(small, k, v, near)
    q = _randn((1, 1, 32, D), torch.float16, 3)
    far = _attend(q, pool, _ints([ids]), _ints([250]))
    ref = _attend(q, small, _ints([[0, 1, 2, 3]]), _ints([250]))
    assert torch.equal(far[0], ref[0]) and torch.equal(far[1], ref[1])
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    kvq.paged_gather(small, near, k2, v2)
    assert torch.equal(kb, k2) and torch.equal(vb, v2)


def test_attention_refusals():
    pages = torch.zeros(4, 2, 10240, dtype=torch.uint8, device="cuda")
    q, table, lens = torch.zeros(3, 8, 128, dtype=torch.float16, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), _ints([1, 2, 3])
    out = torch.empty_like(q)
    bad = [dict(q=q.float()), dict(q=q[..., :64]), dict(q=q[:, :7], out=out[:, :7].contiguous()), dict(out=out[:2]),
           dict(out=out.bfloat16()), dict(table=table.long()), dict(table=table[:2]), dict(lens=lens[:2]),
           dict(lens=lens.long()), dict(pages=pages[:, 0]), dict(pages=pages.cpu()), dict(lse=torch.empty(3, 8, dtype=torch.float16, device="cuda")),
           dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), dict(window=-1), dict(scale=float("inf")),
           dict(lens=lens.cpu()), dict(workspace=torch.empty(64, dtype=torch.uint8)), dict(q=q.transpose(0, 1)),
           dict(table=table.t().contiguous().t())]
    for kw in bad:
        a = dict(q=q, pages=pages, table=table, lens=lens, out=out)
        a.update(kw)
        with pytest.raises((ValueError, kvq.KvqError)):
            kvq.paged_attention(a.pop("q"), a.pop("pages"), a.pop("table"), a.pop("lens"), a.pop("out"), **a)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_is_held_as_nan(D, rotate, dt):
    """A NaN makes its group of 32 channels NaN (a rotated one its partner's as well) and
    nothing else."""
    T, H = 70, 3
    k, v, slots = _randn((T, H, D), dt, 1), _randn((T, H, D), dt, 2), torch.arange(T).int().cuda()
    kw = dict(plan=kvq.RopePlan(D), positions=slots) if rotate else {}
    got = []
    for bad in (float("nan"), 0.0):
        kx, vx = k.clone(), v.clone()
        kx[5, 1, 7], kx[64, 2, D - 1], vx[6, 2, 33], vx[7, 0, 3], vx[7, 0, 60] = (bad,) * 5
        pages = torch.zeros(2, H, kvq.paged_page_bytes(D), dtype=torch.uint8, device="cuda")
        kvq.paged_append(pages, kx, vx, slots, **kw)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        kvq.paged_gather(pages, slots, kb, vb)
        got.append((kb, vb))
    kn, vn = torch.zeros(T, H, D, dtype=torch.bool), torch.zeros(T, H, D, dtype=torch.bool)
    kn[5, 1, 0:32] = kn[64, 2, D - 32:] = vn[6, 2, 32:64] = vn[7, 0, 0:64] = True
    if rotate:
        kn[5, 1, D // 2:D // 2 + 32] = kn[64, 2, D // 2 - 32:D // 2] = True
    for a, b, n in zip(got[0], got[1], (kn.cuda(), vn.cuda())):
        assert torch.equal(a.isnan(), n) and torch.equal(a[~n], b[~n]) and not b.isnan().any()


@pytest.mark.parametrize("layout,rd", [("half", 64), ("half", 40), ("half", 26), ("interleaved", 64), ("interleaved", 36)])
def test_infinities_behind_the_rotated_elements(layout, rd):
    """Elements that no rotation touches are held as without one, infinite ones as 65504."""
    k, slots = _randn((5, 2, 128), torch.float16, 1), _ints([0, 1, 2, 3, 4])
    k[1, 0, 70], k[2, 1, 127] = float("inf"), float("-inf")
    got = []
    for kw in (dict(plan=kvq.RopePlan(128, rotary_dim=rd, layout=layout), positions=slots), {}):
        pages = torch.zeros(1, 2, 10240, dtype=torch.uint8, device="cuda")
        kvq.paged_append(pages, k, k, slots, **kw)
        kb, vb = torch.empty_like(k), torch.empty_like(k)
        kvq.paged_gather(pages, slots, kb, vb)
        got.append((kb, vb))
    assert torch.equal(got[0][0][..., 64:], got[1][0][..., 64:]) and torch.equal(got[0][1], got[1][1])
    assert not got[0][0].isnan().any() and got[0][0][1, 0, 70] > 60000 and got[0][0][2, 1, 127] < -60000


@pytest.mark.parametrize("D,Q,n_rep", [(128, 1, 4), (128, 2, 2), (128, 2, 4), (128, 4, 4), (64, 4, 1), (64, 4, 2), (64, 4, 4)])
@pytest.mark.parametrize("token,window", [(69, 0), (68, 0), (10, 58), (10, 0)])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("columns", [2, 9000])     # (9000: tiles of 16 rows for more than eight)
def test_nan_reaches_the_queries_that_see_it(D, Q, n_rep, token, window, what, columns):
    N, H = 70, 2
    k, v, slots = _randn((N, H, D), torch.float16, 1), _randn((N, H, D), torch.float16, 2), torch.arange(N).int().cuda()
    q = _randn((1, Q, H * n_rep, D), torch.float16, 3)
    got = []
    for bad in (float("nan"), 0.0):
        kx, vx = k.clone(), v.clone()
        (kx if what == "k" else vx)[token, 1, 40] = bad
        pages = torch.zeros(2, H, kvq.paged_page_bytes(D), dtype=torch.uint8, device="cuda")
        kvq.paged_append(pages, kx, vx, slots)
        got.append(_attend(q, pages, _ints(_widened(np.array([[0, 1]], np.int32), columns).tolist()), _ints([N]), window=window))
    (a, la, _), (b, lb, _) = got
    assert not b.isnan().any()
    for i in range(Q):
        end = N - Q + 1 + i
        sees = token < end and (not window or token >= end - window)
        r = slice(n_rep, 2 * n_rep)      # the rows of KV head 1
        assert torch.equal(a[0, i, :n_rep], b[0, i, :n_rep]) and torch.equal(la[0, i, :n_rep], lb[0, i, :n_rep])
        if sees:
            assert (a[0, i, r] if what == "k" else a[0, i, r, 32:64]).isnan().all()
        else:
            assert torch.equal(a[0, i, r], b[0, i, r]) and torch.equal(la[0, i, r], lb[0, i, r])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Q,n_rep", [(1, 4), (2, 4), (3, 5)])      # tiles of 4, 8 and 16 rows
def test_attention_of_2048_sequences(D, Q, n_rep):
    """The largest batch, over shared pages; the arrival counters are zero again behind it."""
    B, g = 2048, np.random.default_rng(D + Q)
    pages = P.make_pages(g.normal(size=(40, 64, D)), g.normal(size=(40, 64, D))).reshape(40, 1, -1)
    kv = P.values(P.unpack(pages, D), D)
    table = g.integers(0, 40, (B, 3)).astype(np.int32)
    lens = g.integers(0, 193, B)
    lens[::97], lens[5] = 0, 192
    q = _randn((B, Q, n_rep, D), torch.float16, 4)
    out, lse, ws = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens.tolist()))
    _check_attention(out, lse, q, kv, table, lens, 0, None)
    assert not ws[:4096].any()


@pytest.mark.parametrize("columns", [4, 9000])
def test_attention_of_4096_rows(columns):
    """64 query tokens of 64 heads on one KV head."""
    pages, table, kv = _cache([200], 1, 128, seed=3)
    q = _randn((1, 64, 64, 128), torch.bfloat16, 4)
    wide = torch.from_numpy(_widened(table, max(columns, table.shape[1]))).cuda()
    out, lse, ws = _attend(q, torch.from_numpy(pages).cuda(), wide, _ints([200]))
    _check_attention(out, lse, q, kv, table, [200], 0, None)
    assert not ws[:4096].any()


def test_empty_calls():
    plan = kvq.RopePlan(128)
    x, n = torch.empty(0, 8, 128, dtype=torch.float16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    pages = torch.zeros(1, 8, 10240, dtype=torch.uint8, device="cuda")
    assert kvq.rope(x, n, plan).shape == x.shape
    kvq.paged_append(pages, x, x, n, positions=n, plan=plan, q=x, q_out=x)
    kvq.paged_gather(pages, n, x, x)
    kvq.paged_attention(x, pages, torch.empty(0, 3, dtype=torch.int32, device="cuda"), n, torch.empty_like(x))
    torch.cuda.synchronize()
    assert not pages.any()


def test_attention_refuses_what_its_positions_cannot_count():
    x = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
    at = x.data_ptr()
    status = kvq.load_library().kvq_paged_attention(0, at, 128, 128, at, 1, at, 1 << 24, 1 << 24, at, 63, 1, 4096, 4096, 128, 0, 0.0,
                                                    at + 4096, None, at, 1 << 30, None)
    assert status == kvq.KVQ_ERR_INVALID and b"too large for one call" in kvq.load_library().kvq_last_error()


# --------------------------------------------------------------------------------------
# streams, graphs, and the operators together
# --------------------------------------------------------------------------------------

def test_two_streams_and_given_streams():
    lens = [900, 65, 300]
    pages, table, kv = _cache(lens, 2, 128, seed=11)
    dev, tab, ln = torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens)
    qs = [_randn((3, 1, 8, 128), torch.float16, s) for s in range(4)]
    want = [_attend(q, dev, tab, ln)[:2] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i, q in enumerate(qs):      # each call with its own workspace, two streams at once
        s = streams[i % 2]
        out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        kvq.paged_attention(q, dev, tab, ln, out, lse=lse, stream=s if i < 2 else s.cuda_stream)
        got.append((out, lse))
    for s in streams:
        s.synchronize()
    for (a, b), (c, d) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, d)


def _step(plan, fused, pages, table, slots, pos, lens, out, ws, Hq, Hkv):
    """One decoding step of one layer: rotate and append, then attend."""
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    kvq.paged_append(pages, k, v, slots, positions=pos, plan=plan, q=q, q_out=q)
    kvq.paged_attention(q, pages, table, lens, out, workspace=ws)


def test_serving_loop_against_64_bits():
    """A prompt per sequence, then decoding steps (one sequence of the batch is padding), as a
    serving loop runs them: append with rotation, attention, read-back; every step's output
    against attention in 64 bits over what the pages hold, and what they hold against the
    rotated keys and values."""
    B, Hq, Hkv, D, steps = 4, 8, 2, 128, 70
    rng = np.random.default_rng(0)
    kw = dict(base=500000.0, scaling="parts", factor=8.0, original_ctx=8192, high=4.0)
    plan = kvq.RopePlan(D, **kw)
    lens = np.array([100, 1, 0, 190])
    order = rng.permutation(40)
    table = order[:B * 10].reshape(B, 10).astype(np.int32)
    pages = torch.zeros(40, Hkv, 10240, dtype=torch.uint8, device="cuda")
    tab = torch.from_numpy(table).cuda()
    ws = torch.zeros(kvq.paged_attention_workspace(B, 1, Hq, Hkv), dtype=torch.uint8, device="cuda")
    # prompts, one flat batch with padding at its end
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)])
    pos = np.concatenate([np.arange(n) for n in lens])
    T = len(seq) + 5
    slots = np.full(T, -1)
    slots[: len(seq)] = table[seq, pos // 64] * 64 + pos % 64
    kp, vp = _randn((T, Hkv, D), torch.float16, 1), _randn((T, Hkv, D), torch.float16, 2)
    posd = _ints(np.r_[pos, np.zeros(5)].astype(int).tolist())
    kr = kvq.rope(kp, posd, plan)
    kvq.paged_append(pages, kp, vp, _ints(slots.tolist()), positions=posd, plan=plan)
    kb, vb = torch.empty_like(kp), torch.empty_like(vp)
    kvq.paged_gather(pages, _ints(slots.tolist()), kb, vb)
    # 4 bits over a group of 32 normal values: half a step of at most (max - min) / 15, about 0.3
    assert float((kb[:len(seq)] - kr[:len(seq)]).abs().max()) <= 0.5 and float((vb[:len(seq)] - vp[:len(seq)]).abs().max()) <= 0.5
    out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")
    for step in range(steps):
        live = lens > 0
        fused = _randn((B, Hq + 2 * Hkv, D), torch.float16, 100 + step)
        raw = fused.clone()
        slots = np.where(live, table[np.arange(B), lens // 64] * 64 + lens % 64, -1)
        pos = np.where(live, lens, 0)
        lens = np.where(live, lens + 1, 0)
        _step(plan, fused, pages, tab, _ints(slots.tolist()), _ints(pos.tolist()), _ints(lens.tolist()), out, ws, Hq, Hkv)
        assert torch.equal(fused[:, :Hq], kvq.rope(raw[:, :Hq], _ints(pos.tolist()), plan))
        assert torch.equal(fused[:, Hq:], raw[:, Hq:])
        if step % 23 == 0 or step == steps - 1:
            kv = P.values(P.unpack(pages.cpu().numpy(), D), D)
            lse = torch.empty(B, Hq, device="cuda")
            again = torch.empty_like(out)
            kvq.paged_attention(fused[:, :Hq], pages, tab, _ints(lens.tolist()), again, lse=lse, workspace=ws)
            assert torch.equal(again, out)
            _check_attention(out, lse, fused[:, None, :Hq], kv, table, lens, 0, None)


def test_captured_and_replayed_step():
    """The step in a CUDA graph: replayed with new inputs, positions and lengths in the same
    buffers it gives what direct calls give; two graphs share a workspace in turn."""
    B, Hq, Hkv, D = 3, 8, 2, 128
    plan = kvq.RopePlan(D)
    lens0, per = [130, 64, 0], 4
    _, table, _ = _cache([256] * B, Hkv, D, seed=1, spare=0)
    table = table[:, :per].copy()
    tab = torch.from_numpy(table).cuda()
    start = torch.zeros(int(table.max()) + 1, Hkv, 10240, dtype=torch.uint8, device="cuda")
    fused = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.float16, device="cuda")
    slots, pos, lens = _ints([-1] * B), _ints([0] * B), _ints([0] * B)
    ws = torch.zeros(kvq.paged_attention_workspace(B, 1, Hq, Hkv), dtype=torch.uint8, device="cuda")
    pages = [start.clone(), start.clone()]
    outs = [torch.zeros(B, Hq, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    _step(plan, fused.clone(), pages[0], tab, slots, pos, lens, outs[0], ws, Hq, Hkv)    # loads the kernels
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(plan, fused, pages[i], tab, slots, pos, lens, outs[i], ws, Hq, Hkv)
        graphs.append(g)
    direct = start.clone()
    out = torch.empty_like(outs[0])
    for step in range(5):
        n = [x + step for x in lens0]
        new = _randn(tuple(fused.shape), torch.float16, step)
        s = [int(table[b, n[b] // 64] * 64 + n[b] % 64) if lens0[b] else -1 for b in range(B)]
        ln = [x + 1 if o else 0 for x, o in zip(n, lens0)]
        for i in range(2):
            fused.copy_(new)
            slots.copy_(_ints(s)), pos.copy_(_ints(n)), lens.copy_(_ints(ln))
            graphs[i].replay()
        _step(plan, new.clone(), direct, tab, _ints(s), _ints(n), _ints(ln), out, ws, Hq, Hkv)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], out) and torch.equal(pages[i], direct)


def test_rope_feeds_the_certified_cache():
    """Rotated queries and keys in the certified cache, as a serving loop of it would do: its
    dense rung equals attention in 64 bits over the rotated keys."""
    N, Hq, Hkv, D = 200, 8, 2, 128
    plan = kvq.RopePlan(D)
    k, v, q = _randn((N, Hkv, D), torch.float16, 1), _randn((N, Hkv, D), torch.float16, 2), _randn((1, Hq, D), torch.float16, 3)
    kr = kvq.rope(k, torch.arange(N).int().cuda(), plan)
    qr = kvq.rope(q, _ints([N - 1]), plan)
    cache = kvq.Cache(1, 1, Hq, Hkv, max_ctx=256)
    try:
        cache.append(0, kr.transpose(0, 1).contiguous()[None], v.transpose(0, 1).contiguous()[None])
        out = torch.empty(1, Hq, D, dtype=torch.float16, device="cuda")
        cache.decode(0, qr, 1.0, 0.25, out)
        torch.cuda.synchronize()
    finally:
        cache.close()
    for h in range(Hkv):
        r = slice(4 * h, 4 * h + 4)
        ref, _, _, _ = P.attention(_f64(qr)[:, r], _f64(kr)[:, h], _f64(v)[:, h], [N], 0, 1 / np.sqrt(D))
        assert np.abs(_f64(out)[:, r] - ref).max() <= 2e-3

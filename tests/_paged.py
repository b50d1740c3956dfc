"""Plain 64-bit definitions of the paged 4-bit cache and of rotary positions (numpy), for
the tests that compare the CUDA calls with them.  The page layout is written out element
by element from include/kvq.h's description, apart from the library's own tables."""

import math

import numpy as np

PAGE, GROUP = 64, 32


# ---- rotary positions ----

def frequencies(rd, base=10000.0, scaling="none", factor=1.0, original_ctx=0, low=1.0, high=32.0):
    """Angle per position of each pair."""
    w = []
    b = base * factor ** (rd / (rd - 2)) if scaling == "ntk" else base
    for i in range(rd // 2):
        x = b ** (-2.0 * i / rd)
        k = 1.0
        if scaling == "linear":
            k = 0.0
        elif scaling == "parts":
            k = (original_ctx * x / (2 * math.pi) - low) / (high - low)
        elif scaling == "yarn":
            d = [rd * math.log(original_ctx / (2 * math.pi * u)) / (2 * math.log(b)) for u in (high, low)]
            lo, hi = max(math.floor(d[0]), 0), min(math.ceil(d[1]), rd - 1)
            k = 1 - (i - lo) / max(hi - lo, 1e-3)
        k = min(1.0, max(0.0, k))
        w.append(x * k + x / factor * (1 - k) if scaling != "ntk" else x)
    return np.array(w)


def rope(x, pos, rd, interleaved, w, magnitude=1.0):
    """[T, H, D] float64 turned by positions [T]."""
    a = np.asarray(pos, np.float64)[:, None, None] * w
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude
    y = np.array(x, np.float64)
    i0, i1 = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    u, v = y[..., i0].copy(), y[..., i1].copy()
    y[..., i0], y[..., i1] = u * c - v * s, v * c + u * s
    return y


# ---- the 4-bit format ----

def _ru16(x):
    """Binary16, rounded up (x >= 0)."""
    h = np.asarray(x, np.float64).astype(np.float16)
    return np.where(h.astype(np.float64) < x, np.nextafter(h, np.float16(np.inf)), h)


def quantize(x, down):
    """[..., D] float64, down [...] bool -> codes [..., D], scale and offset [..., D / 32]
    (binary16) and the quotients that were rounded (for telling near ties)."""
    g = np.clip(x, -65504, 65504).reshape(*x.shape[:-1], -1, GROUP)
    lo, hi, dn = g.min(-1), g.max(-1), np.broadcast_to(np.asarray(down)[..., None], g.shape[:-1])
    o = np.where(dn, hi, lo).astype(np.float16)
    of = o.astype(np.float64)
    s = _ru16(np.maximum(np.where(dn, of - lo, hi - of), 0) / 15)
    sf = s.astype(np.float64)
    d = np.where(dn[..., None], of[..., None] - g, g - of[..., None])
    with np.errstate(divide="ignore", invalid="ignore"):
        quot = np.where(sf[..., None] > 0, d / sf[..., None], 0.0)
    code = np.clip(np.rint(quot), 0, 15)
    return code.reshape(x.shape).astype(np.uint8), np.where(dn, -s, s).astype(np.float16), o, quot.reshape(x.shape)


def page_bytes(D):
    return PAGE * D + 8 * PAGE * (D // GROUP)


def key_code_place(t, c, D):
    g, a, j = c // 32, (c % 32) // 8, c % 8
    return t * (D // 2) + a * 4 * (D // 32) + 4 * g + j // 2, 4 * (j % 2)


def value_code_place(t, c, D):
    g, a, j = c // 32, (c % 32) // 4, c % 4
    byte = a * 2 * (D // 32) + 2 * g + j // 2
    if D == 128:
        return PAGE * D // 2 + (t ^ ((t >> 1) & 1)) * 64 + (byte ^ (32 * ((t >> 2) & 1))), 4 * (j % 2)
    return PAGE * D // 2 + (t ^ ((t >> 2) & 1)) * 32 + byte, 4 * (j % 2)


def scale_places(t, g, D):
    """Bytes of (key scale, key offset, value scale, value offset)."""
    n = D // GROUP
    k = PAGE * D + 2 * (t * n + g)
    v = PAGE * D + 4 * PAGE * n + 2 * (g * PAGE + 16 * ((t >> 1) & 3) + 4 * (t >> 4) + 2 * ((t >> 3) & 1) + (t & 1))
    return k, k + 2 * PAGE * n, v, v + 2 * PAGE * n


_TABLES = {}


def tables(D):
    if D not in _TABLES:
        kb, ks = np.zeros((PAGE, D), int), np.zeros((PAGE, D), int)
        vb, vs = np.zeros((PAGE, D), int), np.zeros((PAGE, D), int)
        sp = np.zeros((4, PAGE, D // GROUP), int)
        for t in range(PAGE):
            for c in range(D):
                kb[t, c], ks[t, c] = key_code_place(t, c, D)
                vb[t, c], vs[t, c] = value_code_place(t, c, D)
            for g in range(D // GROUP):
                sp[:, t, g] = scale_places(t, g, D)
        _TABLES[D] = kb, ks, vb, vs, sp
    return _TABLES[D]


def unpack(raw, D):
    """[..., page bytes] uint8 -> dict of codes [..., 64, D] and scales, offsets
    [..., 64, D / 32] (binary16) of keys and values."""
    kb, ks, vb, vs, sp = tables(D)

    def half(at):
        return (raw[..., at].astype(np.uint16) | (raw[..., at + 1].astype(np.uint16) << 8)).view(np.float16)

    return dict(kc=(raw[..., kb] >> ks) & 15, vc=(raw[..., vb] >> vs) & 15, ks=half(sp[0]), ko=half(sp[1]),
                vs=half(sp[2]), vo=half(sp[3]))


def pack(f, D):
    """The inverse of unpack."""
    kb, ks, vb, vs, sp = tables(D)
    lead = f["kc"].shape[:-2]
    raw = np.zeros((*lead, page_bytes(D)), np.uint8)
    for code, b, s in ((f["kc"], kb, ks), (f["vc"], vb, vs)):
        for sh in (0, 4):
            at = s == sh
            raw[..., b[at]] |= (code[..., at] << sh).astype(np.uint8)
    for name, at in zip(("ks", "ko", "vs", "vo"), sp):
        u = np.ascontiguousarray(f[name]).view(np.uint16)
        raw[..., at], raw[..., at + 1] = u & 255, u >> 8
    return raw


def values(f, D, kind=np.float64):
    """Keys and values that unpacked pages stand for, [..., 64, D]."""
    out = []
    for c, s, o in (("kc", "ks", "ko"), ("vc", "vs", "vo")):
        code = f[c].reshape(*f[c].shape[:-1], D // GROUP, GROUP).astype(kind)
        out.append((code * f[s][..., None].astype(kind) + f[o][..., None].astype(kind)).reshape(f[c].shape))
    return out


def make_pages(k, v):
    """[n, 64, D] float64 keys and values -> [n, page bytes]."""
    D = k.shape[-1]
    odd = np.broadcast_to(np.arange(PAGE) % 2 == 1, k.shape[:-1])
    f = {}
    f["kc"], f["ks"], f["ko"], _ = quantize(k, np.zeros_like(odd))
    f["vc"], f["vs"], f["vo"], _ = quantize(v, odd)
    return pack(f, D)


# ---- attention ----

def attention(q, k, v, ends, window, scale):
    """q [Q, n, D], k, v [N, D] of one KV head (masked tokens' contents are not read), ends
    [Q] tokens that each query sees -> out [Q, n, D], lse [Q, n] and, per query and head, the
    sum of p |v| per channel and the largest scale * sum |q| |k| (for the tolerance)."""
    Q, n, D = q.shape
    out, lse = np.zeros((Q, n, D)), np.full((Q, n), -np.inf)
    pv, qk = np.zeros((Q, n, D)), np.zeros((Q, n))
    for i, end in enumerate(ends):
        lo = max(0, end - window) if window else 0
        if end <= lo:
            continue
        kk, vv = k[lo:end], v[lo:end]
        s = q[i] @ kk.T * scale
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(-1, keepdims=True)
        out[i], pv[i] = p / l @ vv, p / l @ np.abs(vv)
        lse[i] = (m + np.log(l))[:, 0]
        qk[i] = (np.abs(q[i]) @ np.abs(kk).T).max(-1) * scale
    return out, lse, pv, qk

"""Attention weights accumulated per cached token on the GPU, against their definition in 64 bits.

Tolerance: a weight is a sum of p = exp(score - lse).  Scores are within 2^-17 A of the exact ones, A = scale sum |q| (s code +
|o|) <= 3 scale sum |q| max |k^| of a group (as in test_gpu_paged.py's attention), the argument of the exponential is
rounded at a size of at most |score| + |lse| in base 2 (twice 2^-24 of it: the log-sum-exp's own rounding and the sum's),
the exponential is within 2^-22, and sums of n terms within n 2^-24 of their sum: each p is off by at most p (2 (2^-17 A) +
2^-22 (|score| + |lse|) + 2^-21), and what was there before by 2^-23 of it."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402
from test_gpu_paged import TYPES, _f64, _gen, _ints, _randn  # noqa: E402


def _cache(lens, Hkv, D, seed, per=None, kscale=1.0):
    """Pages of keys and values (numpy), and a table of distinct pages in any order; unused entries lie outside."""
    need = [-(-n // 64) for n in lens]
    total = max(1, sum(need))
    rng = np.random.default_rng(seed)
    raw = P.make_pages(rng.standard_normal((total * Hkv, 64, D)) * kscale, rng.standard_normal((total * Hkv, 64, D)))
    table = np.full((len(lens), per or max(1, max(need))), -1, np.int32)
    order, at = rng.permutation(total), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(raw.reshape(total, Hkv, -1)).cuda(), torch.from_numpy(table).cuda()


def _keys(pages, table, b, h, n, D):
    f = P.unpack(pages[table[b, : -(-n // 64)].long().cpu(), h].cpu().numpy() if n else np.zeros((0, P.page_bytes(D)), np.uint8), D)
    return tuple(x.reshape(-1, D)[:n] for x in P.values(f, D))


def _reference(q, lse, pages, table, lens, w, decay, window, scale):
    """The updated weights in 64 bits and their tolerance."""
    B, Q, Hq, D = q.shape
    Hkv = pages.shape[1]
    rep, qf, lf, out = Hq // Hkv, _f64(q), _f64(lse), _f64(w).copy()
    tol = np.abs(out) * 2.0 ** -23
    for b, n in enumerate(lens):
        cols = min(n, w.shape[2])
        if n == 0:
            continue
        t = np.arange(cols)
        for g in range(Hkv):
            k = _keys(pages, table, b, g, n, D)[0][:cols]
            out[b, g, :cols] = 0 if decay == 0 else out[b, g, :cols] * decay
            for i in range(Q):
                hi = n - Q + 1 + i
                lo = max(0, hi - window) if window else 0
                for r in range(g * rep, (g + 1) * rep):
                    if lf[b, i, r] == -np.inf:
                        continue
                    s = (k @ qf[b, i, r]) * scale
                    a = 3 * abs(scale) * np.abs(qf[b, i, r]).sum() * np.abs(k).max(-1)
                    p = np.where((t >= lo) & (t < hi), np.exp(s - lf[b, i, r]), 0.0)
                    out[b, g, :cols] += p
                    tol[b, g, :cols] += p * (2.0 ** -16 * a + 2.0 ** -22 * 1.5 * (np.abs(s) + abs(lf[b, i, r])) + 2.0 ** -21)
            tol[b, g, :cols] += Q * rep * 2.0 ** -23 * np.abs(out[b, g, :cols]) + 2.0 ** -126
    return out, tol


def _lse(q, pages, table, lens, window, scale):
    B, Q, Hq, D = q.shape
    Hkv = pages.shape[1]
    out = np.full((B, Q, Hq), -np.inf)
    for b, n in enumerate(lens):
        for g in range(Hkv):
            k, v = _keys(pages, table, b, g, n, D)
            rows = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            out[b, :, rows] = P.attention(_f64(q)[b, :, rows], k, v, [max(0, n - Q + 1 + i) for i in range(Q)], window, scale)[1]
    return torch.from_numpy(out).float().cuda()


def _run(lens, Q, Hq, Hkv, D, window, decay, dt, seed, per=None, scale=None, kscale=1.0, qscale=1.0):
    pages, table = _cache(lens, Hkv, D, seed, per, kscale)
    q = _randn((len(lens), Q, Hq, D), dt, seed, qscale)
    sc = scale or D ** -0.5
    lse = _lse(q, pages, table, lens, window, sc)
    w = torch.rand(len(lens), Hkv, table.shape[1] * 64, generator=_gen(seed)).cuda()
    before = w.clone()
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w, decay=decay, window=window, scale=scale)
    ref, tol = _reference(q, lse, pages, table, lens, before, decay, window, sc)
    for b, n in enumerate(lens):
        assert torch.equal(w[b, :, n:], before[b, :, n:])
    err = np.abs(_f64(w) - ref)
    assert np.all(err <= tol), float((err - tol).max())
    return w


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,window,decay", [
    ([1], 1, 1, 1, 128, 0, 1.0), ([200, 0, 64, 1, 65], 1, 8, 2, 128, 0, 0.5), ([130, 3], 4, 6, 2, 64, 0, 0.0),
    ([300], 32, 8, 2, 128, 0, 0.0), ([77, 500], 3, 5, 5, 64, 100, 0.9), ([1000], 64, 4, 1, 128, 50, 1.0),
    ([40, 20], 64, 2, 2, 128, 0, 1.0), ([150], 1, 64, 1, 64, 0, -0.5), ([129], 7, 64, 1, 128, 0, 1.0),
    ([700], 1, 3, 3, 128, 1, 1.0)])
def test_weights(lens, Q, Hq, Hkv, D, window, decay, dt):
    _run(lens, Q, Hq, Hkv, D, window, decay, dt, sum(lens) + Q)


@pytest.mark.parametrize("rows", [(64, 64, 128), (33, 64, 64)])
def test_more_rows_than_fit_at_once(rows):
    Q, rep, D = rows
    _run([190, 64], Q, rep, 1, D, 0, 0.7, torch.float16, Q)


@pytest.mark.parametrize("lens,B", [([20000, 5, 9000], 3), (None, 300)])
def test_ranges_over_the_gpu(lens, B):
    """Long and many sequences: pages of a head in several CTAs, and several heads in one."""
    lens = lens or [int(x) for x in np.random.default_rng(5).integers(0, 200, B)]
    _run(lens, 1, 4, 2, 128, 0, 1.0, torch.float16, 17, per=400 if B == 3 else 5)


@pytest.mark.parametrize("qscale,kscale,scale", [(2.0 ** 100, 1.0, 2.0 ** -104), (1e-30, 1.0, 1e29), (1.0, 3e3, 1e-4), (1.0, 1.0, -0.1)])
def test_scales(qscale, kscale, scale):
    _run([150, 70], 2, 4, 2, 128, 0, 1.0, torch.bfloat16, 3, scale=scale, qscale=qscale, kscale=kscale)


def test_sums_of_the_attention():
    """With the attention's own log-sum-exp, each (sequence, KV head)'s weights are Q n_rep in all; 2^-12 for the
    lse's and the weights' errors."""
    lens, Q, Hq, Hkv = [1000, 77, 4], 4, 8, 2
    pages, table = _cache(lens, Hkv, 128, 8)
    q = _randn((3, Q, Hq, 128), torch.bfloat16, 9)
    out, lse = torch.empty_like(q), torch.empty(3, Q, Hq, device="cuda")
    kvq.paged_attention(q, pages, table, _ints(lens), out, lse=lse)
    w = torch.full((3, Hkv, 1024), float("nan"), device="cuda")
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w, decay=0.0)
    for b, n in enumerate(lens):
        assert np.allclose(_f64(w[b, :, :n]).sum(-1), min(Q, n) * Hq / Hkv, rtol=2.0 ** -12)
        assert w[b, :, n:].isnan().all()


def test_operands():
    """Strided queries and weights, entries outside the pool, NaN behind the lengths and in keys, few columns."""
    lens, Q, Hq, Hkv, D = [300, 190], 2, 4, 2, 128
    pages, table = _cache(lens, Hkv, D, 21)
    fused = _randn((2 * Q, Hq + 3, D), torch.float16, 22)
    q = fused[:, 1:1 + Hq].unflatten(0, (2, Q))
    lse = _lse(q, pages, table, lens, 0, D ** -0.5)
    wide = torch.rand(Hkv, 2, 400, generator=_gen(1)).cuda()
    w, keep = wide.transpose(0, 1)[..., 3:3 + 290], wide.clone()
    lost = table[0, 2].item()
    table[0, 2] = 10 ** 6                 # tokens 128..191 are not seen: they only decay
    # sequence 0's last ten tokens have no column: its queries are the last two of 300 all the same
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w, decay=0.5)
    table[0, 2] = lost
    ref, tol = _reference(q, lse, pages, table, lens, keep.transpose(0, 1)[..., 3:3 + 290], 0.5, 0, D ** -0.5)
    before = _f64(keep.transpose(0, 1)[..., 3:3 + 290])
    ref[0, :, 128:192] = before[0, :, 128:192] * 0.5
    assert np.all(np.abs(_f64(w) - ref) <= tol)
    assert torch.equal(wide[..., :3], keep[..., :3]) and torch.equal(wide[..., 293:], keep[..., 293:])


def test_nan():
    lens, D = [100], 128
    pages, table = _cache(lens, 1, D, 31)
    q = _randn((1, 2, 2, D), torch.float16, 1)
    lse = _lse(q, pages, table, lens, 0, D ** -0.5)
    raw = pages.cpu().numpy()
    P_at = P.scale_places(40, 1, D)[1]
    last = int(table[0, 1])
    for t in (100 - 64, 50):                                       # token 100 and on: behind the length
        raw[last, 0, P.scale_places(t, 0, D)[1]:][:2] = 255        # a NaN offset
    raw[int(table[0, 0]), 0, P_at:][:2] = 255                       # token 40's key
    pages = torch.from_numpy(raw).cuda()
    w = torch.zeros(1, 1, 128, device="cuda")
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w)
    bad = w[0, 0].isnan().nonzero()[:, 0].tolist()
    assert bad == [40]
    lse[0, 0, 1] = float("nan")          # the first query sees all but the last token
    w.zero_()
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w)
    assert w[0, 0, :99].isnan().all() and not w[0, 0, 99:].isnan().any()
    lse[0, 0, 1] = float("-inf")
    w.zero_()
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w)
    assert w[0, 0].isnan().nonzero()[:, 0].tolist() == [40]


@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,window", [
    ([1000, 70], 1, 8, 2, 128, 0), ([700], 6, 8, 2, 64, 300), ([900, 130], 10, 8, 2, 128, 0), ([1000], 16, 8, 2, 128, 0), ([900, 300], 33, 8, 2, 64, 500),
    ([2000], 64, 6, 2, 128, 0)])
def test_rows_that_add_nothing_whatever_they_hold(lens, Q, Hq, Hkv, D, window):
    """Rows marked with a log-sum-exp of -inf (padding) whose queries are NaN or infinite, few rows and many, over full pages: the
    same bits as with finite queries there, and the definition's weights.  A KV head of such rows alone is left as it was, also
    where its keys are NaN."""
    pages, table = _cache(lens, Hkv, D, 3)
    q = _randn((len(lens), Q, Hq, D), torch.float16, 4)
    lse = _lse(q, pages, table, lens, window, D ** -0.5)
    rng = np.random.default_rng(Q)
    none = torch.from_numpy(rng.random((len(lens), Q, Hq)) < 0.3).cuda()
    none[0, 0, 0] = True
    none[0, :, Hq // 2:] = True             # KV head 1 of the first sequence
    none[-1, Q - 1, 0] = False
    lse[none] = float("-inf")
    before = torch.rand(len(lens), Hkv, table.shape[1] * 64, generator=_gen(5)).cuda()
    w = before.clone()
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w, decay=1.0, window=window)
    ref, tol = _reference(q, lse, pages, table, lens, before, 1.0, window, D ** -0.5)
    assert np.all(np.abs(_f64(w) - ref) <= tol)
    raw = pages.cpu().numpy()
    for t in (0, 100, 333, 640):            # NaN keys of that KV head, which no row that adds something sees
        at = P.scale_places(t % 64, 1, D)[1]
        raw[int(table[0, t // 64]), 1, at:at + 2] = 255
    bad = q.clone()
    for k, (b, i, r) in enumerate(none.nonzero().tolist()):
        bad[b, i, r, :: 1 + k % D] = (float("nan"), float("inf"), float("-inf"))[k % 3]
    got = before.clone()
    kvq.paged_weights(bad, lse, torch.from_numpy(raw).cuda(), table, _ints(lens), got, decay=1.0, window=window)
    assert torch.equal(got, w) and torch.equal(got[0, 1], before[0, 1])


def test_empty_and_refused_calls():
    pages, table = _cache([100], 2, 64, 1)
    q, lse, lens = _randn((1, 4, 64), torch.float16, 1), torch.zeros(1, 4, device="cuda"), _ints([100])
    w = torch.zeros(1, 2, 128, device="cuda")

    def call(q=q, lse=lse, pages=pages, table=table, lens=lens, w=w, **kw):
        kvq.paged_weights(q, lse, pages, table, lens, w, **kw)

    call(q=q[:0], lse=lse[:0], table=table[:0], lens=lens[:0], w=w[:0])
    for bad in (dict(q=q.float()), dict(lse=lse.double()), dict(lse=lse[:, :3]), dict(w=w.half()), dict(w=w[:, :1]), dict(table=table.long()),
                dict(lens=lens.cpu()), dict(pages=pages[:, :1]), dict(w=w.transpose(1, 2)), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(window=-1), dict(scale=float("inf")), dict(decay=float("nan")), dict(w=w[:, :1].expand(1, 2, 128)), dict(lse=lse.cpu()),
                dict(q=q[:, :3].contiguous(), lse=lse[:, :3].contiguous())):
        with pytest.raises(kvq.KvqError):
            call(**bad)
    torch.cuda.synchronize()
    assert not w.any()


def test_captured_and_on_a_given_stream():
    lens = [700, 90]
    pages, table = _cache(lens, 2, 128, 41)
    q = _randn((2, 1, 8, 128), torch.bfloat16, 5)
    lse, dl = _lse(q, pages, table, lens, 0, 128 ** -0.5), _ints(lens)
    w = torch.zeros(2, 2, 704, device="cuda")
    kvq.paged_weights(q, lse, pages, table, dl, w)
    once, side, graph = w.clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        kvq.paged_weights(q, lse, pages, table, dl, w, decay=0.5)
    w.copy_(once)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, torch.where(once > 0, once * 0.5 + once, once)) or np.allclose(_f64(w), 1.5 * _f64(once), rtol=2.0 ** -22)
    w.zero_()
    torch.cuda.synchronize()
    kvq.paged_weights(q, lse, pages, table, dl, w, stream=side)
    side.synchronize()
    assert torch.equal(w, once)

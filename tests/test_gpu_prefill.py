"""Attention of prompts and chunks over the paged 4-bit cache on the GPU, against its definition in 64 bits.

Tolerances.  Keys enter the tensor cores rounded to binary16 (half a step: 2^-11 of each), so that a score is off by at most
D = (2^-11 + 2^-17) A + 2^-20 with A = scale sum |q| |k| of the row's worst token (2^-17 A: fp32 accumulation and what a
bfloat16 query loses to binary16; 2^-20: roundings of the exponent's argument).  A weight is then off by e^(2D) - 1 (its score
and the sum it is divided by), 2^-11 for its own rounding to binary16 and 2^-11 for the value's:
  out   |out| eps/2 + TINY + (e^(2D) - 1 + 2 2^-11 + 2^-17) sum p |v|, and n 2^-34 max |v| for the weights that count as 0
  lse   D + 2^-21 (|lse| + 1) + n 2^-34
(2^-24 max |v|-sized binary16 subnormals of values lie below TINY's and |v|'s terms: 2^-25 each, added to `tiny`.)"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402
from test_gpu_paged import HALF, TINY, TYPES, _f64, _gen, _ints, _randn  # noqa: E402
from test_gpu_weights import _cache, _keys  # noqa: E402


def _ends(n, m, causal):
    return [max(0, n - m + 1 + i) if causal else n for i in range(m)]


def _check(out, lse, q, starts, pages, table, lens, causal, window, scale, heads=None):
    T, Hq, D = q.shape
    Hkv, dt = pages.shape[1], q.dtype
    rep, qf, of = Hq // Hkv, _f64(q), _f64(out)
    for b, n in enumerate(lens):
        s0, s1 = starts[b], starts[b + 1]
        if s1 <= s0:
            continue
        for g in heads or range(Hkv):
            rows = slice(g * rep, (g + 1) * rep)
            k, v = _keys(pages, table, b, g, n, D)
            ref, rl, pv, a = P.attention(qf[s0:s1, rows], k, v, _ends(n, s1 - s0, causal), window, scale)
            d = (2.0 ** -11 + 2.0 ** -17) * np.abs(a)[..., None] + 2.0 ** -20
            vmax = np.abs(v).max() if n else 0.0
            tol = np.abs(ref) * HALF[dt] + TINY[dt] + 2.0 ** -25 + (np.expm1(2 * d) + 2.0 ** -10 + 2.0 ** -17) * pv + n * 2.0 ** -34 * vmax
            err = np.abs(of[s0:s1, rows] - ref)
            assert np.all(err <= tol), (b, g, float((err - tol).max()), np.argwhere(~(err <= tol))[:3])
            if lse is not None:
                gl = _f64(lse)[s0:s1, rows]
                none = np.isneginf(rl)
                assert np.array_equal(np.isneginf(gl), none)
                lt = d[..., 0] + 2.0 ** -21 * (np.abs(np.where(none, 0, rl)) + 1) + n * 2.0 ** -34
                assert np.all(np.abs(np.where(none, 0, gl) - np.where(none, 0, rl)) <= lt), (b, g)


def _run(lens, chunks, Hq, Hkv, D, dt, causal=True, window=0, scale=None, seed=1, qscale=1.0, kscale=1.0, lead=0, per=None):
    pages, table = _cache(lens, Hkv, D, seed, per, kscale)
    starts = [lead + sum(chunks[:b]) for b in range(len(lens) + 1)]
    T = starts[-1] + lead
    q = _randn((T, Hq, D), dt, seed + 1, qscale)
    out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), out, lse=lse, causal=causal, window=window, scale=scale)
    _check(out, lse, q, starts, pages, table, lens, causal, window, scale or D ** -0.5)
    for x in (out, lse):       # rows of no chunk
        assert (x[:starts[0]] == 7).all() and (x[starts[-1]:] == 7).all()
    again = torch.zeros_like(out)
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), again, causal=causal, window=window, scale=scale)
    assert torch.equal(again[starts[0]:starts[-1]], out[starts[0]:starts[-1]])      # the same bits each time, with and without lse
    return out, lse


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,chunks,Hq,Hkv,D,causal,window", [
    ([1], [1], 1, 1, 128, True, 0), ([5], [5], 4, 1, 64, True, 0), ([64], [64], 4, 2, 128, True, 0), ([128, 65], [128, 1], 2, 2, 64, True, 0),
    ([200], [3], 8, 2, 128, True, 0), ([300, 0, 64, 1, 700], [130, 0, 0, 1, 65], 6, 2, 128, True, 0),
    ([513], [513], 3, 1, 64, True, 0), ([257], [257], 5, 1, 128, True, 100), ([900, 40], [333, 40], 7, 1, 64, True, 64),
    ([700], [129], 4, 2, 128, True, 1), ([300, 77, 0], [300, 50, 0], 4, 2, 128, False, 0), ([130], [1], 12, 3, 64, False, 0),
    ([1500], [70], 64, 1, 128, True, 0), ([2100, 900], [700, 900], 4, 1, 64, True, 500), ([640], [256], 16, 4, 128, True, 0),
    ([1000], [1], 1, 1, 128, True, 0), ([383], [383], 1, 1, 128, False, 0)])
def test_prefill(lens, chunks, Hq, Hkv, D, causal, window, dt):
    _run(lens, chunks, Hq, Hkv, D, dt, causal, window, seed=sum(lens), lead=3)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 24, 3)])
def test_a_long_chunk(D, Hq, Hkv):
    """Ranges over the whole GPU, cut anywhere: 500 tokens behind 3000."""
    lens, chunks = [3500, 100, 2000], [500, 100, 37]
    pages, table = _cache(lens, Hkv, D, 5)
    starts = [0, 500, 600, 637]
    q = _randn((637, Hq, D), torch.bfloat16, 6)
    out, lse = torch.zeros_like(q), torch.zeros(637, Hq, device="cuda")
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), out, lse=lse)
    _check(out, lse, q, starts, pages, table, lens, True, 0, D ** -0.5, heads=[0, Hkv - 1])


def test_a_long_cache():
    """Few rows over 30000 tokens: a row's pieces in many CTAs, and a window that starts within a page."""
    for window in (0, 12345):
        _run([30000], [5], 4, 1, 128, torch.float16, True, window, seed=3)


def test_many_sequences():
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 260, 400)]
    chunks = [int(rng.integers(0, n + 1)) for n in lens]
    _run(lens, chunks, 2, 1, 64, torch.float16, seed=9, per=6)


def test_2048_sequences_of_one_token():
    lens = [1 + b % 5 for b in range(2048)]
    _run(lens, [1] * 2048, 2, 2, 64, torch.bfloat16, seed=10)


@pytest.mark.parametrize("qscale,kscale,scale", [(2.0 ** 100, 1.0, 2.0 ** -104), (1e-30, 1.0, 1e29), (1.0, 3e3, 1e-4), (1.0, 1.0, -0.1),
                                                 (8.0, 4.0, None), (0.0, 1.0, None)])
def test_scales(qscale, kscale, scale):
    _run([300, 70], [150, 70], 4, 2, 128, torch.bfloat16, scale=scale, qscale=qscale, kscale=kscale)


def test_scores_that_grow_and_fall():
    """Rows whose maximum moves up at every page, and down."""
    for up in (1, -1):
        n, D = 900, 64
        rng = np.random.default_rng(3)
        k, v = rng.standard_normal((15, 64, D)) * 0.1, rng.standard_normal((15, 64, D))
        k[..., 0] += (up * np.arange(15 * 64) / 20).reshape(15, 64)
        pages = torch.from_numpy(P.make_pages(k, v)[:, None]).cuda()
        table = torch.arange(15).int().cuda()[None]
        q = _randn((200, 2, D), torch.float16, 4)
        q[..., 0] = 8.0
        out, lse = torch.zeros_like(q), torch.zeros(200, 2, device="cuda")
        kvq.paged_prefill(q, _ints([0, 200]), pages, table, _ints([n]), out, lse=lse)
        _check(out, lse, q, [0, 200], pages, table, [n], True, 0, D ** -0.5)


@pytest.mark.parametrize("D", [64, 128])
def test_elements_at_the_end_of_binary16(D):
    """Keys and values of +-65504, whose held form o + s code may lie beyond it: they are binary16's largest, not infinite."""
    rng = np.random.default_rng(D)
    k = rng.choice([-65504.0, 65504.0, 30000.0], (2, 64, D))
    pages = torch.from_numpy(P.make_pages(k, k[::-1].copy())[:, None]).cuda()
    q = _randn((100, 2, D), torch.bfloat16, 1, 2.0 ** -16)
    out = torch.zeros_like(q)
    kvq.paged_prefill(q, _ints([0, 100]), pages, _ints([0, 1])[None], _ints([128]), out)
    _check(out, None, q, [0, 100], pages, _ints([0, 1])[None], [128], True, 0, D ** -0.5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top", [65504.0, 64992.0, 40000.0])
def test_elements_at_the_end_of_binary16_and_fp16_rows(D, top):
    """The same for rows of fp16, with their log-sum-exp, up to the end and short of it."""
    rng = np.random.default_rng(D)
    k = rng.choice([-top, top, 30000.0], (2, 64, D))
    pages = torch.from_numpy(P.make_pages(k, k[::-1].copy())[:, None]).cuda()
    q, scale = _randn((100, 2, D), torch.float16, 1, 2.0 ** -8), 2.0 ** -8 * D ** -0.5
    out, lse = torch.zeros_like(q), torch.zeros(100, 2, device="cuda")
    kvq.paged_prefill(q, _ints([0, 100]), pages, _ints([0, 1])[None], _ints([128]), out, lse=lse, scale=scale)
    _check(out, lse, q, [0, 100], pages, _ints([0, 1])[None], [128], True, 0, scale)


def test_chunks_that_are_longer_than_their_sequence():
    """The first queries then see nothing: out 0, lse -inf.  Causal, without, and with a window."""
    for causal, window in ((True, 0), (False, 0), (True, 9)):
        out, lse = _run([20, 0], [50, 7], 4, 2, 128, torch.float16, causal, window, seed=7)
        if causal:
            assert not out[:30].any() and lse[:30].isneginf().all()
        assert not out[50:].any() and lse[50:].isneginf().all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens,chunks,D,causal,window", [
    ([20, 0], [50, 7], 128, True, 0), ([20, 0], [50, 7], 64, False, 0), ([300, 0, 5], [400, 3, 40], 128, True, 0), ([300, 1], [400, 300], 64, True, 9),
    ([0] * 400, [1] * 400, 64, True, 0)])
def test_rows_that_see_nothing_whatever_they_hold(lens, chunks, D, causal, window, dt):
    """Padding that holds NaN or infinities: out 0, lse -inf, and the other rows' bits as ever; in units that one CTA writes
    (128 tokens or fewer) and in ones that are merged from pieces."""
    pages, table = _cache(lens, 2, D, 7)
    starts = [sum(chunks[:b]) for b in range(len(lens) + 1)]
    q = _randn((starts[-1], 4, D), dt, 8)
    sees = torch.zeros(starts[-1], dtype=torch.bool)
    for b, n in enumerate(lens):
        sees[starts[b]:starts[b + 1]] = torch.tensor(_ends(n, chunks[b], causal)) > 0
    want, wl = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), want, lse=wl, causal=causal, window=window)
    none = (~sees).nonzero()[:, 0].tolist()
    for k, t in enumerate(none):
        q[t, k % 4] = (float("nan"), float("inf"), float("-inf"))[k % 3]
        q[t, (k + 1) % 4, k % D] = (float("inf"), float("-inf"), float("nan"))[k % 3]
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), out, lse=lse, causal=causal, window=window)
    assert not out[none].any() and lse[none].isneginf().all()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    if sees.any():          # and one that sees its sequence's first token alone, or all
        t = int(sees.nonzero()[0])
        q[t, 2, 5] = float("-inf")
        kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), out, lse=lse, causal=causal, window=window)
        assert out[t, 2].isnan().all() and lse[t, 2].isnan()
        out[t, 2], lse[t, 2] = want[t, 2], wl[t, 2]
        assert torch.equal(out, want) and torch.equal(lse, wl)
    table.fill_(2 ** 30)    # no page of the pool: no token is seen
    q[:, 1] = float("nan")
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), out, lse=lse, causal=causal, window=window)
    assert not out.any() and lse.isneginf().all()


def test_operands():
    """A view of a fused projection, a padded table, entries outside the pool, starts that run backwards or out of the rows."""
    lens, Hq, Hkv, D = [300, 190], 4, 2, 128
    pages, table = _cache(lens, Hkv, D, 21, per=9)
    fused = _randn((150, Hq + 4, D), torch.float16, 22)
    q, starts = fused[:, 2:2 + Hq], [0, 100, 150]
    out = torch.zeros(150, Hq, D, dtype=torch.float16, device="cuda")
    kvq.paged_prefill(q, _ints(starts), pages, table[:, :5], _ints(lens), out)
    _check(out, None, q, starts, pages, table, lens, True, 0, D ** -0.5)
    want = out.clone()
    # tokens 64..127 of the second sequence are in no page of the pool: not seen
    table[1, 1] = 2 ** 30
    kvq.paged_prefill(q, _ints(starts), pages, table, _ints(lens), out)
    assert torch.equal(out[:100], want[:100])
    few = torch.cat([table[1:, :1], table[1:, 2:]], 1).contiguous()          # the sequence without them
    lse = torch.zeros(50, Hq, device="cuda")
    short = torch.zeros(50, Hq, D, dtype=torch.float16, device="cuda")
    kvq.paged_prefill(q[100:], _ints([0, 50]), pages, few, _ints([126]), short, lse=lse)
    _check(out[100:], None, q[100:], [0, 50], pages, few, [126], True, 0, D ** -0.5)
    # beyond the rows: cut off; backwards: empty
    for bad in ([0, 100, 10 ** 9], [-5, 100, 150], [-2 ** 31, 2 ** 31 - 1, -7]):
        kvq.paged_prefill(q, _ints(bad), pages, table, _ints(lens), torch.empty_like(out))
    torch.cuda.synchronize()


@pytest.mark.parametrize("end", [-2 ** 31, -2 ** 31 + 1, -2 ** 30, -1])
def test_starts_at_the_ends_of_their_range(end):
    """Starts far below 0 are clamped to 0 like any other: ascending ones are chunks as ever, and behind a start above them they
    leave an empty chunk (the difference of unclamped ends would wrap to 2^31 - 100 rows at -2^31)."""
    lens, Hq, Hkv, D = [300, 190, 77], 4, 2, 128
    pages, table = _cache(lens, Hkv, D, 21)
    q = _randn((150, Hq, D), torch.float16, 22)
    out, lse = torch.full_like(q, 7.0), torch.full((150, Hq), 7.0, device="cuda")
    kvq.paged_prefill(q, _ints([0, 100, end, end]), pages, table, _ints(lens), out, lse=lse)
    assert (out[100:] == 7).all() and (lse[100:] == 7).all()
    kvq.paged_prefill(q, _ints([end, end, end, 100]), pages, table, _ints(lens), out.fill_(7), lse=lse.fill_(7))
    _check(out, lse, q, [0, 0, 0, 100], pages, table, lens, True, 0, D ** -0.5)
    assert (out[100:] == 7).all() and (lse[100:] == 7).all()


def test_offsets_beyond_32_bits():
    """A pool of 5 GB, the sequence's pages at its end."""
    n_pages, Hkv, D = 70000, 8, 128
    pages = torch.empty(n_pages, Hkv, P.page_bytes(D), dtype=torch.uint8, device="cuda")
    small, table = _cache([200], Hkv, D, 2)
    pages[-4:] = small
    q = _randn((70, 8, D), torch.float16, 3)
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    kvq.paged_prefill(q, _ints([0, 70]), small, table, _ints([200]), want)
    kvq.paged_prefill(q, _ints([0, 70]), pages, table + (n_pages - 4), _ints([200]), out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("token,window", [(69, 0), (150, 0), (10, 58), (199, 0), (0, 0)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_reaches_the_queries_that_see_it(D, token, window, what):
    n, m, Hq = 200, 150, 2
    pages, table = _cache([n], 1, D, 5)
    raw = pages.cpu().numpy()
    at = P.scale_places(token % 64, 1, D)[1 if what == "k" else 3]
    clean = torch.from_numpy(raw.copy()).cuda()
    raw[int(table[0, token // 64]), 0, at:at + 2] = 255
    last = raw[int(table[0, 3]), 0]
    for t in range(n - 192, 64):          # behind the length
        for o in P.scale_places(t, 0, D):
            last[o:o + 2] = 255
    pages, q = torch.from_numpy(raw).cuda(), _randn((m, Hq, D), torch.float16, 6)
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    lse, wl = torch.zeros(m, Hq, device="cuda"), torch.zeros(m, Hq, device="cuda")
    kvq.paged_prefill(q, _ints([0, m]), clean, table, _ints([n]), want, lse=wl, window=window)
    kvq.paged_prefill(q, _ints([0, m]), pages, table, _ints([n]), out, lse=lse, window=window)
    ends = np.array(_ends(n, m, True))
    sees = torch.from_numpy((token < ends) & ((token >= ends - window) if window else True)).cuda()
    assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wl[~sees])
    assert out[sees][..., 32:64].isnan().all()
    if what == "k":
        assert out[sees].isnan().all() and lse[sees].isnan().all()


@pytest.mark.parametrize("D,lens,chunks,causal,window", [
    (128, [200, 90], [150, 90], True, 0), (64, [200, 90], [150, 90], True, 58), (128, [3000, 700], [300, 64], True, 0),
    (64, [3000, 700], [300, 64], False, 0), (128, [5000], [3], True, 2000), (64, [130] * 40, [130] * 40, True, 100)])
def test_nan_values_reach_their_channels_alone(D, lens, chunks, causal, window):
    """Values that are NaN in one group: those channels of the queries that see the token, in whole units and in pieces; other
    channels and lse have the same bits as without, and so have weights that go by that lse."""
    Hq, Hkv = 4, 2
    pages, table = _cache(lens, Hkv, D, 5)
    raw, rng = pages.cpu().numpy(), np.random.default_rng(sum(lens))
    hit = [sorted({0, n // 2, n - 1, int(rng.integers(0, n))}) for n in lens]
    for b, ts in enumerate(hit):
        for t in ts:
            at = P.scale_places(t % 64, t % (D // 32), D)[3]
            raw[int(table[b, t // 64]), 1, at:at + 2] = 255             # of KV head 1
    starts = [sum(chunks[:b]) for b in range(len(lens) + 1)]
    q = _randn((starts[-1], Hq, D), torch.float16, 6)
    got = []
    for pool in (pages, torch.from_numpy(raw).cuda()):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        kvq.paged_prefill(q, _ints(starts), pool, table, _ints(lens), out, lse=lse, causal=causal, window=window)
        got.append((out, lse))
    (want, wl), (out, lse) = got
    assert torch.equal(lse, wl)
    bad = torch.zeros_like(out, dtype=torch.bool)
    for b, ts in enumerate(hit):
        ends = np.array(_ends(lens[b], chunks[b], causal))
        for t in ts:
            sees = (t < ends) & ((t >= ends - window) if window else True)
            gr = t % (D // 32)
            bad[starts[b]:starts[b + 1], Hq // 2:, 32 * gr:32 * gr + 32] |= torch.from_numpy(sees).cuda()[:, None, None]
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], want[~bad])
    Q = min(chunks)
    ends = _ints(starts)[1:].long()[:, None] - Q + torch.arange(Q, device="cuda")
    if causal and Q <= 64:
        w = torch.zeros(2, len(lens), Hkv, table.shape[1] * 64, device="cuda")
        for k, x in enumerate((wl, lse)):
            kvq.paged_weights(q[ends], x[ends].contiguous(), pages, table, _ints(lens), w[k], window=window)
        assert torch.equal(w[0], w[1]) and not w.isnan().any()


def test_queries_that_are_nan_or_infinite():
    """... make their own rows NaN, and no others."""
    pages, table = _cache([300], 1, 128, 5)
    q = _randn((150, 2, 128), torch.bfloat16, 6)
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    kvq.paged_prefill(q, _ints([0, 150]), pages, table, _ints([300]), want)
    q[3, 1, 7], q[140, 0, 100] = float("nan"), float("inf")
    kvq.paged_prefill(q, _ints([0, 150]), pages, table, _ints([300]), out)
    bad = torch.zeros(150, 2, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[140, 0] = True
    assert torch.equal(out[~bad], want[~bad]) and out[bad].isnan().all()


def test_against_the_decode_attention():
    """The same rows by both calls: each within its own tolerance of the definition, so both within their sum."""
    lens, Q, Hq, Hkv, D = [700, 65, 200], 4, 8, 2, 128
    pages, table = _cache(lens, Hkv, D, 12)
    q = _randn((3, Q, Hq, D), torch.bfloat16, 13)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    la, lb = torch.zeros(3, Q, Hq, device="cuda"), torch.zeros(3, Q, Hq, device="cuda")
    kvq.paged_attention(q, pages, table, _ints(lens), a, lse=la)
    kvq.paged_prefill(q.flatten(0, 1), _ints([0, 4, 8, 12]), pages, table, _ints(lens), b.flatten(0, 1), lse=lb.flatten(0, 1))
    assert (a.float() - b.float()).abs().max() <= 2 * 2.0 ** -8 * 4 + 2.0 ** -7
    assert (la - lb).abs().max() <= 2.0 ** -10 * 64


def test_empty_and_refused_calls():
    pages, table = _cache([100], 2, 64, 1)
    q, lens, starts = _randn((10, 4, 64), torch.float16, 1), _ints([100]), _ints([0, 10])
    out, lse = torch.full_like(q, 7.0), torch.zeros(10, 4, device="cuda")

    def call(q=q, starts=starts, pages=pages, table=table, lens=lens, out=out, **kw):
        return kvq.paged_prefill(q, starts, pages, table, lens, out, **kw)

    call(q=q[:0], out=out[:0])
    call(starts=starts[:1], table=table[:0], lens=lens[:0])
    call(starts=_ints([4, 4]))
    for bad in (dict(q=q.float()), dict(out=out.bfloat16()), dict(out=out[:9]), dict(out=out.transpose(0, 1)), dict(starts=starts[:1]),
                dict(starts=starts.long()), dict(starts=starts.cpu()), dict(lens=lens.cpu()), dict(table=table.long()), dict(pages=pages[0]),
                dict(lse=lse.half()), dict(lse=lse[:, :2]), dict(workspace=lse), dict(q=q[0]), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(window=-1), dict(window=5, causal=False), dict(scale=float("nan")), dict(out=q), dict(lse=lse.cpu()), dict(q=q[:, :3], out=out[:, :3].contiguous()),
                dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(kvq.KvqError):
            call(**bad)
    torch.cuda.synchronize()
    assert (out == 7).all()


def test_two_streams_and_replayed_graphs():
    """Two calls at once, each with its own workspace; two graphs that share one, replayed in turn with other lengths."""
    lens, Hq, Hkv, D = [900, 300], 8, 2, 128
    pages, table = _cache(lens, Hkv, D, 31)
    q = _randn((200, Hq, D), torch.bfloat16, 32)
    starts, dl = _ints([0, 150, 200]), _ints(lens)
    want = torch.zeros_like(q)
    kvq.paged_prefill(q, starts, pages, table, dl, want)
    outs, streams = [torch.zeros_like(q) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(kvq.paged_prefill_workspace(200, 2, Hq, Hkv, D), dtype=torch.uint8, device="cuda").fill_(255) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, s, w in zip(outs, streams, ws):
            kvq.paged_prefill(q, starts, pages, table, dl, o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    kvq.paged_prefill(q, starts, pages, table, dl, outs[0].zero_(), stream=streams[0])      # its own workspace
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for k, (gr, o) in enumerate(zip(graphs, outs)):
        with torch.cuda.graph(gr):
            kvq.paged_prefill(q, starts, pages, table, dl, o, window=100 * k, workspace=ws[0])
    for other in ([900, 300], [700, 50], [150, 50]):
        dl.copy_(_ints(other))
        for k, (gr, o) in enumerate(zip(graphs, outs)):
            gr.replay()
            torch.cuda.synchronize()
            _check(o, None, q, [0, 150, 200], pages, table, other, True, 100 * k, D ** -0.5)

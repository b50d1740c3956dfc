"""The paged cache's calls together, as a serving loop uses them: prompts of an image and text with positions on three axes
are appended in chunks and attend over the pages, their last queries say what the cache keeps, it is cut back, and decoding
goes on over what is left.  Each step is compared with its definition in 64 bits on what the pages hold at that point
(tolerances: test_gpu_prefill.py, test_gpu_weights.py and test_gpu_paged.py)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402
from test_gpu_paged import _f64, _gen, _ints, _randn  # noqa: E402
from test_gpu_evict import kept  # noqa: E402
from test_gpu_prefill import _check  # noqa: E402
from test_gpu_weights import _keys, _reference  # noqa: E402


def _grid(T, seed):
    """Time, height, width of T tokens: text, then an image of 12 x 17 patches, then text again."""
    t = np.arange(T)
    img = (t >= 30) & (t < 30 + 204)
    k = t - 30
    pos = np.stack([np.where(img, 30, np.where(t < 30, t, t - 187)), np.where(img, 30 + k // 17, np.where(t < 30, t, t - 187)),
                    np.where(img, 30 + k % 17, np.where(t < 30, t, t - 187))])
    return torch.from_numpy(pos.astype(np.int32)).cuda()


@pytest.mark.parametrize("D,dt", [(128, torch.bfloat16), (64, torch.float16)])
def test_prompt_to_bounded_cache_to_decoding(D, dt):
    Hq, Hkv, lens, keep, first, recent = 8, 2, [700, 333], 200, 4, 40
    B, rep, per = 2, 4, 12
    plan = kvq.RopePlan(D, base=1000000.0, axes=(D // 8, 3 * D // 16, 3 * D // 16), axis_order="cycled")
    pool = torch.zeros(40, Hkv, kvq.paged_page_bytes(D), dtype=torch.uint8, device="cuda")
    order = torch.randperm(40, generator=_gen(1)).int()
    table = order[: B * per].reshape(B, per).cuda().contiguous()
    new_table = order[B * per: B * per + 2 * 6].reshape(B, 6).cuda().contiguous()
    done, chunk = [0] * B, 256
    outs = []
    while any(d < n for d, n in zip(done, lens)):
        m = [min(chunk, n - d) for d, n in zip(done, lens)]
        starts = [0, m[0], m[0] + m[1]]
        T = starts[-1]
        fused = _randn((T, Hq + 2 * Hkv, D), dt, sum(done) + 5)
        q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        pos = torch.cat([_grid(lens[b], b)[:, done[b]:done[b] + m[b]] for b in range(B)], 1).contiguous()
        at = [torch.arange(done[b], done[b] + m[b]) for b in range(B)]
        slots = torch.cat([table[b].cpu()[a // 64] * 64 + a % 64 for b, a in enumerate(at)]).int().cuda()
        kvq.paged_append(pool, k, v, slots, positions=pos, plan=plan, q=q, q_out=q)
        done = [d + x for d, x in zip(done, m)]
        out, lse = torch.zeros(T, Hq, D, dtype=dt, device="cuda"), torch.zeros(T, Hq, device="cuda")
        kvq.paged_prefill(q, _ints(starts), pool, table, _ints(done), out, lse=lse)
        _check(out, lse, q, starts, pool, table, done, True, 0, D ** -0.5)
        outs.append((q.clone(), lse, starts, list(done)))
    # the last 16 queries of each prompt: the first prompt's come from the last chunk, the second's from its own last one
    Q = 16
    last = [next((c, o) for o in reversed(outs) for c in [o[2][b + 1] - o[2][b]] if c >= Q) for b in range(B)]
    qw = torch.stack([o[0][o[2][b + 1] - Q:o[2][b + 1]] for b, (_, o) in enumerate(last)])
    lw = torch.stack([o[1][o[2][b + 1] - Q:o[2][b + 1]] for b, (_, o) in enumerate(last)])
    assert [o[3][b] for b, (_, o) in enumerate(last)] == lens
    w = torch.full((B, Hkv, per * 64), float("nan"), device="cuda")
    kvq.paged_weights(qw, lw, pool, table, _ints(lens), w, decay=0.0)
    ref, tol = _reference(qw, lw, pool, table, lens, torch.zeros_like(w), 0.0, 0, D ** -0.5)
    for b, n in enumerate(lens):
        assert np.all(np.abs(_f64(w)[b, :, :n] - ref[b, :, :n]) <= tol[b, :, :n])
        # the sums of softmax rows whose log-sum-exp is the prefill's: within its 2^-11 of the scores' size (|score| < 2^4)
        assert np.allclose(_f64(w)[b, :, :n].sum(-1), Q * rep, rtol=2.0 ** -7)
    # cut back, each KV head to its own tokens
    held = [[_keys(pool, table, b, g, n, D) for g in range(Hkv)] for b, n in enumerate(lens)]
    new_lens, new_w = _ints([0, 0]), torch.zeros(B, Hkv, 6 * 64, device="cuda")
    origin = kvq.paged_evict(pool, table, _ints(lens), w, new_table, new_lens, keep, first=first, recent=recent, new_weights=new_w)
    assert new_lens.tolist() == [keep, keep]
    wn, on = w.cpu().numpy(), origin.cpu().numpy()
    for b, n in enumerate(lens):
        for g in range(Hkv):
            ids = kept(wn[b, g], n, keep, first, recent)
            assert np.array_equal(on[b, g], ids)
            for x, y in zip(_keys(pool, new_table, b, g, keep, D), held[b][g]):
                assert np.array_equal(x, y[ids])
    # decoding: append behind what is kept, attend, accumulate; the positions go on where the prompts ended
    for step in range(3):
        n = keep + step + 1
        q, k, v = _randn((B, Hq, D), dt, 50 + step), _randn((B, Hkv, D), dt, 60 + step), _randn((B, Hkv, D), dt, 70 + step)
        pos = _ints([[lens[b] - 187 + step for b in range(B)]] * 3)
        slot = _ints([int(new_table[b, (n - 1) // 64]) * 64 + (n - 1) % 64 for b in range(B)])
        kvq.paged_append(pool, k, v, slot, positions=pos, plan=plan, q=q, q_out=q)
        out, lse = torch.zeros_like(q), torch.zeros(B, Hq, device="cuda")
        kvq.paged_attention(q, pool, new_table, _ints([n, n]), out, lse=lse)
        before = new_w.clone()
        kvq.paged_weights(q, lse, pool, new_table, _ints([n, n]), new_w, decay=0.9)
        ref, tol = _reference(q[:, None], lse[:, None], pool, new_table, [n, n], before, 0.9, 0, D ** -0.5)
        assert np.all(np.abs(_f64(new_w) - ref) <= tol)
        for b in range(B):
            for g in range(Hkv):
                rows = slice(g * rep, (g + 1) * rep)
                kk, vv = _keys(pool, new_table, b, g, n, D)
                want, _, pv, a = P.attention(_f64(q)[b, None, rows], kk, vv, [n], 0, D ** -0.5)
                eps = 2.0 ** -11 if dt is torch.float16 else 2.0 ** -8
                # test_gpu_paged.py: (2 (2^-17 3A) + 2^-17) sum p |v| beside the output's rounding
                assert np.all(np.abs(_f64(out)[b, None, rows] - want) <= np.abs(want) * eps + 2.0 ** -24 + (6 * 2.0 ** -17 * a[..., None] + 2.0 ** -17) * pv)
    # a second eviction, of what the first one left and what came behind it, back into the first pages
    again, back = table[:, :4].contiguous(), _ints([0, 0])
    origin = kvq.paged_evict(pool, new_table, _ints([keep + 3] * 2), new_w, again, back, 100, first=first, recent=recent)
    wn, on = new_w.cpu().numpy(), origin.cpu().numpy()
    for b in range(B):
        for g in range(Hkv):
            ids = kept(wn[b, g], keep + 3, 100, first, recent)
            assert np.array_equal(on[b, g], ids)
            for x, y in zip(_keys(pool, again, b, g, 100, D), _keys(pool, new_table, b, g, keep + 3, D)):
                assert np.array_equal(x, y[ids])


def test_a_captured_step():
    """Prefill of a chunk, weights and eviction in one graph, replayed with other data."""
    Hq, Hkv, D, n, m = 4, 1, 64, 300, 70
    plan = kvq.RopePlan(D, axes=(8, 12, 12))
    pool = torch.zeros(12, Hkv, kvq.paged_page_bytes(D), dtype=torch.uint8, device="cuda")
    table, new_table = _ints([[3, 1, 7, 2, 5]]), _ints([[8, 9]])
    K, V = _randn((n, Hkv, D), torch.float16, 1), _randn((n, Hkv, D), torch.float16, 2)
    t = torch.arange(n)
    slots = (table[0].cpu()[t // 64] * 64 + t % 64).int().cuda()
    pos, q = torch.stack([t, t // 7, t % 7]).int().cuda(), _randn((m, Hq, D), torch.float16, 3)
    starts, lens, new_lens = _ints([0, m]), _ints([n]), _ints([0])
    out, lse = torch.zeros_like(q), torch.zeros(m, Hq, device="cuda")
    w, origin = torch.zeros(1, Hkv, 320, device="cuda"), torch.zeros(1, Hkv, 100, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvq.paged_prefill_workspace(m, 1, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def step():
        kvq.paged_append(pool, K, V, slots, positions=pos, plan=plan)
        kvq.paged_prefill(q, starts, pool, table, lens, out, lse=lse, workspace=ws)
        kvq.paged_weights(q[-8:][None], lse[-8:][None], pool, table, lens, w, decay=0.0)
        kvq.paged_evict(pool, table, lens, w, new_table, new_lens, 100, recent=8, origin=origin)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (11, 12):
        for x, s in ((K, seed), (V, seed + 5), (q, seed + 9)):
            x.copy_(_randn(x.shape, torch.float16, s))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, lse, w[..., :n], origin)]
        _check(out, lse, q, [0, m], pool, table, [n], True, 0, D ** -0.5)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, w[..., :n], origin)))

"""Eviction from the paged cache by weight on the GPU: which tokens are kept, against a sort in numpy, and where their
bytes go.  Everything is exact: indices, weights and codes, scales and offsets are moved, not computed."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402
from test_gpu_paged import _gen, _ints  # noqa: E402


def kept(w, n, keep, first, recent):
    """Indices that a head keeps of n tokens with weights w."""
    if n <= keep:
        return np.arange(n)
    rest = np.arange(first, n - recent)
    x = w[rest].astype(np.float64)
    x = np.where(np.isnan(x), np.inf, x)
    order = np.lexsort((rest, -x, ~np.isnan(w[rest])))       # a NaN first, then the largest, then the lowest index
    return np.sort(np.r_[np.arange(first), rest[order[: keep - first - recent]], np.arange(n - recent, n)])


def _case(lens, Hkv, D, seed, spare=2):
    """A pool of random bytes, a table of distinct pages, and a table of other ones."""
    need = [-(-max(n, 0) // 64) for n in lens]
    per = max(1, max(need))
    total = sum(need) + sum(max(1, n) for n in need) + spare
    pages = torch.randint(0, 256, (total, Hkv, P.page_bytes(D)), generator=_gen(seed)).to(torch.uint8).cuda()
    order = torch.randperm(total, generator=_gen(seed + 1)).int()
    table = torch.full((len(lens), per), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table.cuda(), order[at:].clone()


def _free(order, B, per):
    return order[: B * per].reshape(B, per).cuda().contiguous()


def _bits(raw, D):
    """Codes and the bits of scales and offsets of pages as numpy."""
    f = P.unpack(raw.cpu().numpy(), D)
    return {n: x.view(np.uint16) if x.dtype == np.float16 else x for n, x in f.items()}


def _check(pages, before, table, lens, w, new_table, new_lens, keep, first, recent, origin, new_w, D, to=None, to_before=None):
    B, Hkv = w.shape[:2]
    to, to_before = (pages if to is None else to), (before if to is None else to_before)
    src, dst, was = _bits(before, D), _bits(to, D), _bits(to_before, D)
    table, new_table, origin = (x.cpu().numpy() for x in (table, new_table, origin))
    wn, touched = w.cpu().numpy(), np.zeros((to.shape[0], Hkv, 64), bool)
    assert new_lens.cpu().tolist() == [min(max(n, 0), keep) for n in lens]
    for b, n in enumerate(lens):
        n = max(n, 0)
        for h in range(Hkv):
            ids = kept(wn[b, h], n, keep, first, recent)
            m = len(ids)
            assert m == min(n, keep)
            assert np.array_equal(origin[b, h, :m], ids), (b, h)
            assert (origin[b, h, m:] == -1).all()
            if new_w is not None:
                got = new_w[b, h].cpu().numpy()
                assert np.array_equal(got[:m], wn[b, h, ids], equal_nan=True) and (got[m:keep] == 0).all()
            sp, dp = table[b, ids // 64], new_table[b, np.arange(m) // 64]
            ok = (dp >= 0) & (dp < to.shape[0])
            there = (sp >= 0) & (sp < pages.shape[0])
            for f in src:
                want = np.where(there[:, None], src[f][np.where(there, sp, 0), h, ids % 64], 0)
                assert np.array_equal(dst[f][dp[ok], h, (np.arange(m) % 64)[ok]], want[ok]), (f, b, h)
            touched[dp[ok], h, (np.arange(m) % 64)[ok]] = True
    for f in src:       # everything else is as it was
        assert np.array_equal(dst[f][~touched], was[f][~touched]), f


@pytest.mark.parametrize("lens,Hkv,D,keep,first,recent", [
    ([100], 1, 128, 64, 0, 0), ([1, 0, 64, 65, 130], 2, 64, 64, 3, 5), ([1100, 999, 1000, 1001], 8, 128, 1000, 4, 128),
    ([200, 77], 3, 128, 1, 0, 0), ([200, 77], 3, 64, 1, 1, 0), ([200, 77], 3, 64, 1, 0, 1), ([300], 2, 128, 128, 64, 64),
    ([5000, 4097], 2, 64, 4096, 0, 100), ([20000, 3, 16385], 1, 128, 777, 10, 33), ([40000], 2, 64, 30001, 0, 0),
    ([-3, 70], 1, 128, 65, 0, 7)])
def test_evict(lens, Hkv, D, keep, first, recent):
    pages, table, order = _case(lens, Hkv, D, len(lens) + keep)
    B, per = len(lens), -(-keep // 64)
    if len(order) < B * per:
        order = torch.arange(pages.shape[0], pages.shape[0] + B * per).int()
        pages = torch.cat([pages, torch.zeros(B * per, *pages.shape[1:], dtype=torch.uint8, device="cuda")])
    N = max(1, table.shape[1] * 64)
    w = torch.exp(2 * torch.randn(B, Hkv, N, generator=_gen(keep))).cuda()
    w[..., 5::7] = 0                                            # many that are equal
    w[..., 3::11] = 0.25
    new_table, new_lens = _free(order, B, per), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    new_w = torch.full((B, Hkv, keep + 5), 7.0, device="cuda")
    before = pages.clone()
    origin = kvq.paged_evict(pages, table, _ints(lens), w, new_table, new_lens, keep, first=first, recent=recent, new_weights=new_w)
    _check(pages, before, table, lens, w, new_table, new_lens, keep, first, recent, origin, new_w, D)
    assert (new_w[..., keep:] == 7).all()


@pytest.mark.parametrize("n", [130, 9000])
def test_weights_of_every_kind(n):
    """Negative ones, infinities, NaN, both zeros, subnormals; all equal."""
    keep, Hkv = 100, 6
    pages, table, order = _case([n], Hkv, 64, n)
    w = torch.randn(1, Hkv, table.shape[1] * 64, generator=_gen(2))
    w[0, 0, ::3] = float("inf")
    w[0, 1, 5::9], w[0, 1, 3::2] = float("nan"), float("-inf")
    w[0, 2] = 0.0
    w[0, 2, 1::2] = -0.0
    w[0, 3] = -1e-42 * torch.arange(w.shape[-1])
    w[0, 4] = float("nan")
    w[0, 5] = torch.where(w[0, 5] > 0, 1.0, float("-inf"))
    w = w.cuda()
    new_table, new_lens, before = _free(order, 1, 2), _ints([0]), pages.clone()
    new_w = torch.zeros(1, Hkv, keep, device="cuda")
    origin = kvq.paged_evict(pages, table, _ints([n]), w, new_table, new_lens, keep, first=2, recent=3, new_weights=new_w)
    _check(pages, before, table, [n], w, new_table, new_lens, keep, 2, 3, origin, new_w, 64)


def test_long_row():
    """Slices of a row that do not fit into shared memory (300000 tokens), and its 128K prefix."""
    n, Hkv, keep = 300000, 1, 5000
    pages = torch.randint(0, 256, (5000, Hkv, P.page_bytes(64)), generator=_gen(3)).to(torch.uint8).cuda()
    table = torch.arange(n // 64 + 1).int().cuda()[None] % 4800
    w = torch.rand(1, Hkv, table.shape[1] * 64, generator=_gen(4)).cuda()
    w[0, 0, 1000:200000] = 0.5          # the border lies among equal ones
    for m in (n, 131072):
        new_table, new_lens, before = (4800 + torch.arange(79)).int().cuda()[None], _ints([0]), pages.clone()
        origin = kvq.paged_evict(pages, table, _ints([m]), w, new_table, new_lens, keep, first=1, recent=4000)
        _check(pages, before, table, [m], w, new_table, new_lens, keep, 1, 4000, origin, None, 64)


def test_operands():
    """Strided weights and tables, another pool, entries outside the pools, columns fewer than tokens."""
    lens, Hkv, D, keep = [300, 250, 40], 2, 128, 130
    pages, table, order = _case(lens, Hkv, D, 11)
    table[1, 1] = pages.shape[0] + 3
    wide = torch.rand(Hkv, 3, 1000, generator=_gen(5)).cuda()
    w = wide.transpose(0, 1)[..., 7:7 + 290]                    # 290 columns: sequence 0 counts as 290 tokens
    to = torch.randint(0, 256, (12, Hkv, P.page_bytes(D)), generator=_gen(6)).to(torch.uint8).cuda()
    tables = torch.full((3, 9), -1, dtype=torch.int32)
    tables[:, :3] = torch.tensor([[0, 5, 2], [7, 100, 3], [9, 4, 1]])
    tables, new_lens, before, to_before = tables.cuda(), _ints([0, 0, 0]), pages.clone(), to.clone()
    new_w = torch.zeros(3, Hkv, 200, device="cuda")
    origin = torch.empty(3, Hkv, keep, dtype=torch.int32, device="cuda")
    got = kvq.paged_evict(pages, table, _ints(lens), w, tables[:, :3], new_lens, keep, first=4, recent=30, origin=origin,
                          new_weights=new_w, new_pages=to)
    assert got is origin and torch.equal(pages, before)
    _check(pages, before, table, [290, 250, 40], w, tables[:, :3], new_lens, keep, 4, 30, origin, new_w, D, to, to_before)


def test_empty_and_refused_calls():
    pages, table, order = _case([100], 2, 64, 1)
    w, lens, out = torch.rand(1, 2, 128, device="cuda"), _ints([100]), _ints([0])
    new_table = _free(order, 1, 1)

    def call(keep=64, pages=pages, table=table, lens=lens, w=w, new_table=new_table, out=out, **kw):
        return kvq.paged_evict(pages, table, lens, w, new_table, out, keep, **kw)

    before = pages.clone()
    none = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    call(table=none, lens=_ints([]), w=w[:0], new_table=none, out=_ints([]))
    for bad in (dict(w=w.double()), dict(w=w[:, :1]), dict(w=w.transpose(1, 2)), dict(lens=lens.long()), dict(out=out.cpu()),
                dict(table=table.long()), dict(new_table=new_table[0]), dict(origin=torch.empty(1, 2, 63, dtype=torch.int32, device="cuda")),
                dict(new_weights=torch.zeros(1, 2, 63, device="cuda")), dict(pages=pages[..., :-1]), dict(stream=torch.cuda.current_stream())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(keep=65), dict(keep=0), dict(first=-1), dict(recent=65), dict(first=33, recent=32), dict(new_table=table),
                dict(out=lens), dict(new_weights=w), dict(new_weights=torch.zeros(1, 1, 64, device="cuda").expand(1, 2, 64))):
        with pytest.raises(kvq.KvqError):
            call(**bad)
    torch.cuda.synchronize()
    assert torch.equal(pages, before)


def test_captured_and_replayed_on_another_stream():
    lens = [500, 130]
    pages, table, order = _case(lens, 2, 128, 21)
    w = torch.rand(2, 2, 512, device="cuda")
    new_table, new_lens = _free(order, 2, 3), _ints([0, 0])
    origin, dl = torch.empty(2, 2, 150, dtype=torch.int32, device="cuda"), _ints(lens)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    before = pages.clone()
    with torch.cuda.graph(graph, stream=side):
        kvq.paged_evict(pages, table, dl, w, new_table, new_lens, 150, recent=9, origin=origin)
    for k in range(3):
        w.copy_(torch.rand(2, 2, 512, generator=_gen(k)))
        graph.replay()
        torch.cuda.synchronize()
        _check(pages, before, table, lens, w, new_table, new_lens, 150, 0, 9, origin, None, 128)
    kvq.paged_evict(pages, table, dl, w, new_table, new_lens, 150, recent=9, origin=origin, stream=side)
    side.synchronize()
    _check(pages, before, table, lens, w, new_table, new_lens, 150, 0, 9, origin, None, 128)

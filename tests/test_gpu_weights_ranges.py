"""Accumulated attention weights on the GPU where a CTA goes over many tiles and heads, from few query rows of a KV head to more
than the kernels hold at once, against the definition in 64 bits (tolerances: test_gpu_weights.py).

A GPU of 152 SMs takes a call's pages (or tiles of two) in as many equal ranges: 8 KV heads of 20000 tokens are 1256 tiles, 8
per CTA, which is more than its buffers and accumulators in flight; 120 sequences of 4 heads are three heads per CTA."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
from test_gpu_paged import _f64, _gen, _ints, _randn  # noqa: E402
from test_gpu_weights import _cache, _lse, _reference  # noqa: E402


def _check(lens, Q, rep, Hkv, D, window, decay, dt, seed, columns=None, hole=None):
    pages, table = _cache(lens, Hkv, D, seed)
    q = _randn((len(lens), Q, rep * Hkv, D), dt, seed)
    lse = _lse(q, pages, table, lens, window, D ** -0.5)
    before = torch.rand(len(lens), Hkv, columns or table.shape[1] * 64, generator=_gen(seed)).cuda()
    if hole is not None:                 # an entry outside the pool: its tokens only decay
        b0, page = hole
        kept, table[b0, page] = table[b0, page].item(), 2 ** 30
    w = before.clone()
    kvq.paged_weights(q, lse, pages, table, _ints(lens), w, decay=decay, window=window)
    for b in sorted({0, len(lens) // 2, len(lens) - 1}):      # a sequence by itself, its ranges cut elsewhere: the same bits
        one = before[b:b + 1].clone()
        kvq.paged_weights(q[b:b + 1], lse[b:b + 1], pages, table[b:b + 1], _ints(lens[b:b + 1]), one, decay=decay, window=window)
        assert torch.equal(one[0], w[b])
    if hole is not None:
        table[b0, page] = kept
    ref, tol = _reference(q, lse, pages, table, lens, before, decay, window, D ** -0.5)
    if hole is not None:
        at = slice(64 * page, min(64 * page + 64, ref.shape[2], lens[b0]))
        ref[b0, :, at] = _f64(before)[b0, :, at] * decay
    err = np.abs(_f64(w) - ref)
    assert np.all(err <= tol), (float((err - tol).max()), np.argwhere(~(err <= tol))[:4])
    for b, n in enumerate(lens):
        assert torch.equal(w[b, :, n:], before[b, :, n:])


ROWS = [(6, 4), (10, 4), (14, 4), (19, 3), (16, 4), (32, 4), (43, 3), (50, 5)]     # 24, 40, 56, 57, 64, 128, 129, 250 rows


@pytest.mark.parametrize("Q,rep", ROWS)
@pytest.mark.parametrize("D,dt", [(128, torch.float16), (64, torch.bfloat16)])
def test_long_sequences(Q, rep, D, dt):
    """Many tiles of a head in one CTA, heads that end within a range, a page outside the pool."""
    _check([20000, 3001], Q, rep, 4, D, 0, 0.5, dt, Q + D, hole=(0, 100))


@pytest.mark.parametrize("Q,rep", ROWS)
def test_windows_and_columns(Q, rep):
    """Pages before a window in the middle of ranges, tokens without a column."""
    _check([20000, 9000], Q, rep, 4, 64, 4321, 1.0, torch.float16, Q, columns=15000)


@pytest.mark.parametrize("Q,rep", ROWS)
@pytest.mark.parametrize("D", [64, 128])
def test_many_short_sequences(Q, rep, D):
    """Several sequences and heads per CTA, empty ones among them, some shorter than their queries."""
    lens = [int(x) for x in np.random.default_rng(Q).integers(0, 260, 120)]
    lens[7] = lens[8] = lens[119] = 0
    _check(lens, Q, rep, 2 if D == 128 else 4, D, 0, 0.0 if D == 64 else 0.9, torch.float16, Q)


@pytest.mark.parametrize("Q,rep,D", [(16, 4, 128), (64, 4, 64), (14, 4, 128)])
def test_eight_heads_of_a_long_sequence(Q, rep, D):
    _check([20037], Q, rep, 8, D, 0, 1.0, torch.bfloat16, 9)

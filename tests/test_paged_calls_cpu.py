"""Refusals of the paged prefill, weights and eviction calls that come before any CUDA call, and their no-ops."""

import ctypes

import pytest

import certified_quantized_kv_gb300 as kvq

ADDR = 1 << 20                 # addresses that are never read
A, B, C, D, E, F, G = (ADDR + (k << 16) for k in range(7))


def _error():
    return kvq.load_library().kvq_last_error()


def prefill(**kw):
    a = dict(dtype=0, q=A, qt=4096, qh=128, starts=B, T=10, pages=C, n_pages=5, table=D, ts=4, max_pages=4, lens=E, batch=2, Hq=32,
             Hkv=8, hd=128, causal=1, window=0, scale=0.0, out=F, lse=None, ws=G, nbytes=1 << 40)
    a.update(kw)
    return kvq.load_library().kvq_paged_prefill(*a.values(), None)


def weights(**kw):
    a = dict(dtype=0, q=A, qt=4096, qh=128, lse=B, pages=C, n_pages=5, table=D, ts=4, max_pages=4, lens=E, batch=2, Q=1, Hq=32, Hkv=8,
             hd=128, window=0, scale=0.0, decay=1.0, w=F, ws=2048, wh=256, cols=256)
    a.update(kw)
    return kvq.load_library().kvq_paged_weights(*a.values(), None)


def evict(**kw):
    a = dict(pages=A, n_pages=5, table=B, ts=4, max_pages=4, lens=C, batch=2, Hkv=8, hd=128, w=D, ws=2048, wh=256, cols=256, keep=100,
             first=4, recent=20, to=A, to_pages=5, new_table=E, nts=2, new_max=2, new_lens=F, origin=G, nw=None, nws=0, nwh=0)
    a.update(kw)
    return kvq.load_library().kvq_paged_evict(*a.values(), None)


SHARED = [(dict(n_pages=0), b"n_pages"), (dict(n_pages=(1 << 25) + 1), b"n_pages"), (dict(max_pages=0), b"max_pages"),
          (dict(max_pages=1 << 24, batch=2048), b"max_pages"), (dict(ts=-1), b"stride"), (dict(batch=-1), b"batch"),
          (dict(batch=2049), b"batch"), (dict(Hkv=0), b"n_kv_heads"), (dict(Hkv=4097), b"n_"), (dict(hd=96), b"head_dim")]
ROWS = [(dict(dtype=2), b"dtype"), (dict(Hq=33), b"n_q_heads"), (dict(Hq=8 * 65), b"n_q_heads"), (dict(window=-1), b"window"),
        (dict(scale=float("nan")), b"scale"), (dict(scale=2.9e38), b"scale"), (dict(qt=4), b"q: strides"), (dict(qh=-8), b"q: strides")]


@pytest.mark.parametrize("call", [prefill, weights, evict])
@pytest.mark.parametrize("bad,word", SHARED)
def test_shapes(call, bad, word):
    assert call(**bad) == kvq.KVQ_ERR_INVALID and word in _error() and b"kvq_paged_" + call.__name__.encode() in _error()


@pytest.mark.parametrize("call", [prefill, weights])
@pytest.mark.parametrize("bad,word", ROWS)
def test_rows(call, bad, word):
    assert call(**bad) == kvq.KVQ_ERR_INVALID and word in _error()


@pytest.mark.parametrize("bad,word", [(dict(T=-1), b"n_tokens"), (dict(T=(1 << 24) + 1), b"n_tokens"), (dict(causal=2), b"causal"),
                                      (dict(causal=0, window=5), b"window"), (dict(out=A), b"out"),
                                      (dict(T=1 << 24, Hq=64 * 4096, Hkv=4096, max_pages=1 << 24, batch=1), b"too large")])
def test_prefill(bad, word):
    assert prefill(**bad) == kvq.KVQ_ERR_INVALID and word in _error()


@pytest.mark.parametrize("bad,word", [(dict(Q=0), b"n_q_tokens"), (dict(Q=65), b"n_q_tokens"), (dict(cols=0), b"column"),
                                      (dict(decay=float("inf")), b"decay"), (dict(wh=255), b"overlap"), (dict(ws=100), b"overlap"),
                                      (dict(ws=-2048), b"overlap")])
def test_weights(bad, word):
    assert weights(**bad) == kvq.KVQ_ERR_INVALID and word in _error()


@pytest.mark.parametrize("bad,word", [(dict(keep=0), b"keep"), (dict(keep=129), b"keep"), (dict(new_max=0), b"keep"), (dict(first=-1), b"first"),
                                      (dict(first=81), b"first"), (dict(recent=2 ** 31 - 1), b"recent"), (dict(to_pages=0), b"n_pages"),
                                      (dict(new_table=B), b"page_table"), (dict(new_lens=C), b"seq_lens"), (dict(nts=1), b"new_table"),
                                      (dict(nw=D, nws=800, nwh=100), b"new_weights"), (dict(nw=F, nws=800, nwh=99), b"overlap"),
                                      (dict(cols=0), b"column"), (dict(wh=-1), b"strides")])
def test_evict(bad, word):
    assert evict(**bad) == kvq.KVQ_ERR_INVALID and word in _error()


def test_prefill_counts_chunks_that_overlap():
    """Starts are only read on the device; if they do not ascend each of the chunks can be all of q."""
    big = dict(T=1 << 24, Hq=64 * 512, Hkv=512, max_pages=1 << 18)
    assert prefill(batch=2048, **big) == kvq.KVQ_ERR_INVALID and b"too large" in _error()


def test_no_ops():
    for call in (prefill, weights, evict):
        assert call(batch=0) == kvq.KVQ_OK
    assert prefill(T=0) == kvq.KVQ_OK


def test_workspace_shape():
    n = ctypes.c_size_t()
    lib = kvq.load_library()
    assert lib.kvq_paged_prefill_workspace(10, 1, 32, 8, 128, None) == kvq.KVQ_ERR_INVALID
    for bad in ((-1, 1, 32, 8, 128), (10, 2049, 32, 8, 128), (10, 1, 33, 8, 128), (10, 1, 32, 8, 80)):
        assert lib.kvq_paged_prefill_workspace(*bad, ctypes.byref(n)) == kvq.KVQ_ERR_INVALID
        assert b"kvq_paged_prefill_workspace" in _error()

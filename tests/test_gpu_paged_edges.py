"""The paged 4-bit cache on the GPU at the edges of its number ranges and of its calls.  Definitions and
tolerances are those of tests/test_gpu_paged.py where nothing else is said."""

import os
import shutil
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import certified_quantized_kv_gb300 as kvq  # noqa: E402
import _paged as P  # noqa: E402
from test_gpu_paged import TYPES, _attend, _cache, _check_append, _check_attention, _f64, _gen, _ints, _randn, _widened  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_spans_that_fp32_does_not_hold(D, dt):
    """A large extreme of 15 h (h binary16) beside a tiny one of the other sign: the span passes 15 h by
    less than fp32 shows, and 15 steps of h do not reach over it.  Scales and offsets are exact."""
    T, H, G = 64, 2, D // 32
    tiny = 2.0 ** -24        # in both types and in binary16
    g = _gen(D)
    x = torch.rand(T, H, G, 32, generator=g) * 7 + 1
    h = 2.0 ** torch.randint(0, 5, (T, H, G), generator=g)
    sign = torch.where(torch.rand(T, H, G, generator=g) < 0.5, -1.0, 1.0)
    x[..., 3], x[..., 17] = 15 * h, -tiny
    x = (x * sign[..., None]).reshape(T, H, D).to(dt).cuda()
    pages = torch.zeros(2, H, P.page_bytes(D), dtype=torch.uint8, device="cuda")
    slots = _ints(list(range(20, 20 + T)))
    before = pages.clone()
    kvq.paged_append(pages, x, x, slots)
    _check_append(before, pages, _f64(x), _f64(x), slots, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Q,Hq,columns", [(1, 4, 0), (1, 8, 0), (2, 8, 9000)])      # tiles of 4, 8 and 16 rows
@pytest.mark.parametrize("exponent,scale,kscale", [(124, 2.0 ** -126, 1.0), (118, 2.0 ** -121, 1.0), (-110, 2.0 ** 107, 1.0),
                                                   (-122, 2.0 ** 121, 1.0), (126, 2.0 ** -126, 0.02), (-3, -0.7, 1.0)])
def test_queries_over_the_whole_range_of_bfloat16(exponent, scale, kscale, Q, Hq, columns, D):
    """Rows near the type's largest and smallest numbers whose scores are moderate; at 2^126 all elements have
    one sign, so that the sums over a group of channels pass what fp32 holds."""
    lens = [300, 65]
    pages, table, kv = _cache(lens, 1, D, seed=abs(exponent), kscale=kscale)
    q = torch.randn(2, Q, Hq, D, generator=_gen(D + Q))
    q = (1 + torch.rand(2, Q, Hq, D, generator=_gen(D)) if exponent == 126 else q).double() * 2.0 ** exponent
    q = q.to(torch.bfloat16).cuda()
    assert torch.isfinite(q).all()
    tab = torch.from_numpy(_widened(table, columns) if columns else table).cuda()
    out, lse, _ = _attend(q, torch.from_numpy(pages).cuda(), tab, _ints(lens), scale=scale)
    _check_attention(out, lse, q if scale > 0 else -q, kv, table, lens, 0, abs(scale))


def test_rows_of_any_size_in_one_tile():
    """Four heads of one KV head, 2^-100 to 2^100 times as large: each row has its own power of two."""
    lens, D = [200], 128
    pages, table, kv = _cache(lens, 1, D, seed=6)
    size = torch.tensor([2.0 ** -100, 1.0, 2.0 ** 100, 0.0])[:, None]
    q = (torch.randn(1, 1, 4, D, generator=_gen(8)).double() * size).to(torch.bfloat16).cuda()
    for scale in (2.0 ** -103, 0.11, 2.0 ** 97):
        row = {2.0 ** -103: 2, 0.11: 1, 2.0 ** 97: 0}[scale]
        out, lse, _ = _attend(q, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(), _ints(lens), scale=scale)
        rows = [r for r in range(4) if r == row or r == 3 or size[r, 0] < size[row, 0]]   # (the others' scores pass fp32)
        for r in rows:
            _check_attention(out[:, :, r:r + 1], lse[:, :, r:r + 1], q[:, :, r:r + 1], kv, table, lens, 0, scale)


def _compiled(tmp_path, name, *flags):
    """tests/host/<name>.cu, built against the kernels' headers."""
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / name)
    cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
           os.path.join(ROOT, "certified_quantized_kv_gb300", "csrc"), os.path.join(ROOT, "tests", "host", name + ".cu"), *flags, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def _says_ok(exe):
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-3000:] + r.stderr[-1000:]


def test_pieces_of_a_warp_whose_copy_never_arrived(tmp_path):
    """The merge of an attention call's pieces by itself (tests/host/paged_merge.cu): sums as in 64 bits, and NaN
    rows where a piece may hold anything."""
    _says_ok(_compiled(tmp_path, "paged_merge"))


def test_attention_calls_of_several_host_threads(tmp_path):
    """Threads with batches of their own size, streams and workspaces (tests/host/paged_threads.cu): no call
    takes shared memory away from another one's launch."""
    lib = os.path.dirname(kvq.LIB_PATH)
    _says_ok(_compiled(tmp_path, "paged_threads", "-L", lib, "-l:libkvq.so", "-Xlinker", "-rpath", "-Xlinker", lib))

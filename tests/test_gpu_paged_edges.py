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
from test_gpu_paged import TYPES, _check_append, _f64, _gen, _ints  # noqa: E402

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

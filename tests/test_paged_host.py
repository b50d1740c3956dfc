"""Index arithmetic of the rotary and paged-cache kernels, enumerated on the host: tests/host/paged_host.cu is
compiled with nvcc against the kernels' own headers and run without a GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    exe = str(tmp_path_factory.mktemp("host") / "paged_host")
    cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
           os.path.join(ROOT, "certified_quantized_kv_gb300", "csrc"), os.path.join(ROOT, "tests", "host", "paged_host.cu"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def _run(program, check):
    r = subprocess.run([program, check], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-3000:]


def test_rows_exchange_within_the_room_of_their_warp(program):
    """Rotation of halves that are no multiple of 4: no lane reads outside its warp's shared memory."""
    _run(program, "rows")


def test_a_late_copy_is_waited_for(program):
    """The paged attention's ring after a wait that ran out: the copies in flight are the ones waited for."""
    _run(program, "ring")


def test_overlap_of_rows(program):
    _run(program, "overlap")

"""The benchmark's token-by-token loops run, at a small size: the certified cache with and
without rotated queries and keys, and the paged 4-bit cache."""

import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("flags,mode", [([], "decode_loop"), (["--rope"], "decode_loop"), (["--cache", "paged"], "paged_loop"),
                                        (["--cache", "paged", "--batch", "3"], "paged_loop")])
def test_loop(flags, mode):
    r = subprocess.run([sys.executable, "bench.py", "--loop", "--layers", "2", "--ctx", "1000", "--steps", "3", "--warmup", "3",
                        *flags], cwd=ROOT, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["mode"] == mode and line["value"] > 0 and line["ctx_end"] == 1000

"""The norm and distillation suites again in one child process whose launches
hold 4096 work-items, so that a call over many rows is several launches, each
with its own first row or block."""
import os
import subprocess
import sys

import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_suites_with_split_launches():
    torch_cuda().cuda.empty_cache()
    cmd = [sys.executable, "-u", "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
           "-k", "not offsets_past_32_bits", "tests/test_gpu_norm.py", "tests/test_gpu_distill.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, DDP_MAX_LAUNCH_ITEMS="4096"), capture_output=True,
                       text=True, timeout=300)
    tail = (r.stdout[-4000:] + "\n" + r.stderr[-2000:]).strip()
    assert r.returncode == 0, tail
    assert " passed" in r.stdout

"""The range, token and workspace suites once more against the checked build
(every global index and TMA coordinate range-checked in the kernels)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["tests/test_gpu_chunk_range.py", "tests/test_gpu_quant_range.py",
          "tests/test_gpu_quant_tokens.py", "tests/test_gpu_shared_workspace.py",
          "tests/test_gpu_cluster_room.py"]


def test_range_suites_pass_on_the_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if os.environ.get("DECODE_ATTN_CHECKED") == "1":
        pytest.skip("already running on the checked build")
    env = dict(os.environ, DECODE_ATTN_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-m", "gpu", "-x", "-q",
                        "-p", "no:cacheprovider", *SUITES],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:]
    assert " passed" in r.stdout

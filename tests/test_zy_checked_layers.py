"""The tests of the operators around layers once more, in a child process that
loads the checked build (every global access that a kernel computes is tested
against its buffer): the same results, and no violation recorded; and the
tests of its records."""
import os
import subprocess
import sys

import pytest
import torch

from reducescatter_reduction_gb300 import build as ccl_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("name", ["test_layer_bounds.py", "test_expert_sort.py", "test_expert_rows.py", "test_grads.py", "test_norm_e4m3.py"])
def test_checked_build_passes(name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    env = dict(os.environ, CCL_LIBRARY=ccl_build.build_checked())
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.join(HERE, name)]
    res = subprocess.run(cmd, cwd=os.path.dirname(HERE), env=env, capture_output=True, text=True, timeout=1200)
    tail = (res.stdout + res.stderr)[-3000:]
    assert res.returncode == 0, tail
    assert " passed" in res.stdout and "skipped" not in res.stdout.splitlines()[-1], tail

"""Further tests of the operators on logits in a child process that loads the
checked build: those of its records, and those whose sizes, lists and layouts
reach what test_zy_checked_logits.py does not."""
import os
import subprocess
import sys

import pytest
import torch

from reducescatter_reduction_gb300 import build as ccl_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("name", ["test_logit_bounds.py", "test_logit_in_place.py", "test_rules_biases.py", "test_balance_ranges.py",
                                  "test_logit_limits.py"])
def test_checked_build_passes(name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    env = dict(os.environ, CCL_LIBRARY=ccl_build.build_checked())
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.join(HERE, name)]
    res = subprocess.run(cmd, cwd=os.path.dirname(HERE), env=env, capture_output=True, text=True, timeout=1200)
    tail = (res.stdout + res.stderr)[-3000:]
    assert res.returncode == 0, tail
    assert " passed" in res.stdout and "skipped" not in res.stdout.splitlines()[-1], tail

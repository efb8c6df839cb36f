"""What the logit operators accept at the ends of their arguments' ranges: the
refusals on the CPU, the results there on a GPU."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import rng
from test_logit_refusals import BAD, OK, distill_call, front, status      # noqa: F401 (front: a fixture)


@pytest.mark.cpu
@pytest.mark.parametrize("temperature,want", [
    (1e-45, BAD), (1e-40, BAD), (4.2e-39, BAD), (4.3e-39, OK), (1e-38, OK), (1e-30, OK), (3e38, OK), (-1e-40, BAD)])
def test_temperatures_whose_reciprocal_is_infinite(front, temperature, want):      # noqa: F811
    assert status(front, distill_call(front, temperature=temperature)) == (want, int(want == OK))
    if want == BAD:
        assert b"temperature" in front.fake_message()

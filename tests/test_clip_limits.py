"""ccl_grad_clip takes every finite limit: the largest float is how a caller measures without clipping."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import stream
from test_layer_refusals import BAD, INF, OK, check, front, grads, tensor  # noqa: F401  (front: the fixture)

FLT_MAX = float(np.finfo(np.float32).max)


@pytest.mark.cpu
@pytest.mark.parametrize("max_norm, want", [(FLT_MAX, OK), (3.4e38, OK), (3.401e38, OK), (2.0 ** -149, OK), (0.0, OK), (-2.0 ** -149, BAD), (INF, BAD)])
def test_limits(front, max_norm, want):  # noqa: F811
    check(front, grads(front, "clip", tensor(), max_norm=max_norm), want, "" if want == OK else "max_norm")


@pytest.mark.gpu
@pytest.mark.parametrize("norm, factor", [(5.0, 1.0), (FLT_MAX, 1.0), (INF, 0.0), (0.0, 1.0)])
def test_the_largest_limit_clips_nothing(norm, factor):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.randn(5001, device="cuda")
    out, before, at = torch.empty_like(x), x.clone(), torch.tensor([norm, -1.0], device="cuda")
    h = ccl.ccl_comm_create(1, [x.data_ptr()])
    ccl.ccl_grad_clip(h, [ccl.Tensor(x.data_ptr(), out.data_ptr(), 5001, ccl.CCL_F32, 0)], FLT_MAX, at.data_ptr(), stream())
    ccl.ccl_comm_check(h)
    ccl.ccl_comm_destroy(h)
    assert float(at[1]) == factor and torch.equal(out, before * factor) and torch.equal(x, before)

"""The fused RMSNorm's exchange under wait limits that run out: a CTA that gives up leaves only when the others of its row
have sent their sums, so the call ends, is reported if a wait ran out, and the next one gives the oracle's bits."""
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from reducescatter_reduction_gb300 import inputs
from ccl_testutil import Comm, RankBuffers, ensure_built, stream_ptr
from test_rmsnorm import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


@pytest.mark.parametrize("dtype, p, rows, hidden", [("bf16", 8, 2, 8192), ("f32", 3, 60, 1001), ("bf16", 2, 160, 12288), ("bf16", 8, 330, 16384)])
@pytest.mark.parametrize("limit, stall", [(1, 0), (500, 0), (20000, 0), (1, 1)])
def test_limits_that_run_out(dtype, p, rows, hidden, limit, stall):
    n = rows * hidden
    xs = [inputs.normal(n, 7, r, 0.5, dtype) for r in range(p)]
    res, gamma = inputs.normal(n, 7, 100, 1.0, dtype), inputs.normal(hidden, 7, 200, 1.0, dtype)
    storage = inputs.STORAGE[dtype]
    ins, outs = RankBuffers(xs, n, storage), RankBuffers(None, n, storage, p=p)
    r_in, r_out, g = RankBuffers([res], n, storage), RankBuffers(None, n, storage, p=1), RankBuffers([gamma], hidden, storage)
    with Comm(ins, outs) as cm:
        def call():
            ccl.ccl_allreduce_residual_rmsnorm(cm.h, dtype, rows, hidden, r_in.ptr(0), r_out.ptr(0), g.ptr(0), 1e-6, "ring", stream_ptr())

        ccl.ccl_comm_set_debug(cm.h, limit, stall)
        for _ in range(5):
            call()
            try:
                ccl.ccl_comm_check(cm.h)
                assert not stall
            except ccl.CclError as e:
                assert e.status == ccl.CCL_ERR_TIMEOUT
        ccl.ccl_comm_set_debug(cm.h, 0, 0)
        call()
        torch.cuda.synchronize()
        ccl.ccl_comm_check(cm.h)
    check(outs, r_out, xs, res, gamma, rows, hidden, dtype, "ring")
    for b in (ins, outs, r_in, r_out, g):
        assert b.guards_intact()

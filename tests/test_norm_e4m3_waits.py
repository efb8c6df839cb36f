"""The exchange between the CTAs of a row under wait limits that run out: a CTA that gives up leaves only when the others
of its row have sent what they send, so the call ends, is reported if a wait ran out, and the next one is right."""
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from test_norm_e4m3 import Norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# rows of two to eight CTAs, of each CTA shape
SIZES = [("bf16", 8, 2, 8192, 0), ("f32", 2, 100, 4096, 64), ("bf16", 3, 5, 5001, 0), ("bf16", 2, 200, 33000, 128), ("f16", 5, 300, 65536, 0),
         ("bf16", 1, 400, 33000, 0), ("f32", 4, 310, 40000, 32), ("bf16", 2, 310, 33001, 0)]


def checked(h):
    """Whether the communicator reports a wait that ran out."""
    try:
        ccl.ccl_comm_check(h)
    except ccl.CclError as e:
        assert e.status == ccl.CCL_ERR_TIMEOUT
        return True
    return False


@pytest.mark.parametrize("dtype, p, rows, hidden, group", SIZES)
@pytest.mark.parametrize("limit", [1, 500, 20000])
def test_limits_that_run_out(dtype, p, rows, hidden, group, limit):
    n = Norm(dtype, p, rows, hidden, group)
    h = n.comm.h
    ccl.ccl_comm_set_debug(h, limit, 0)
    for _ in range(5):
        n.call(h)
        if not checked(h):
            n.check()
    ccl.ccl_comm_set_debug(h, 0, 0)
    with n.comm:
        n.call(h)
    n.check()


@pytest.mark.parametrize("dtype, p, rows, hidden, group", SIZES)
def test_sums_that_are_withheld(dtype, p, rows, hidden, group):
    n = Norm(dtype, p, rows, hidden, group)
    h = n.comm.h
    ccl.ccl_comm_set_debug(h, 1, 1)
    n.call(h)
    assert checked(h)
    ccl.ccl_comm_set_debug(h, 0, 0)
    with n.comm:
        n.call(h)
    n.check()

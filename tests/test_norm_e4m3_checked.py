"""The checked build's tests of the accesses of the norm with e4m3 output, each against the row it addresses: with the last
row taken away (the debug hook) every access to it is recorded and not made, and the record names a byte of a row.
These tests run only against the checked library (test_zy_checked_layer_edges.py runs them against it)."""
import os
import re

import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from test_norm_e4m3 import Norm

if "CCL_LIBRARY" not in os.environ:
    pytest.skip("the default build has no bounds checks (CCL_LIBRARY selects the checked build)", allow_module_level=True)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _checked():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ccl.load_library()
    if not ccl.ccl_bounds_checked():
        pytest.skip("the default build has no bounds checks (CCL_LIBRARY selects the checked build)")


def bits(t):
    return t.contiguous().view(torch.uint8)


# one and more CTAs a row, units kept and read again, whole groups and single elements, chunks that end inside rows and units
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("p, rows, hidden, group", [
    (1, 9, 64, 0), (8, 9, 8192, 128), (5, 9, 4104, 0), (2, 9, 1001, 32), (4, 200, 264, 32), (3, 200, 33000, 0), (64, 200, 24, 0), (64, 160, 17, 64),
    (2, 400, 512, 64), (7, 400, 9000, 0), (3, 400, 1001, 64), (1, 400, 33001, 0)])
def test_the_record_names_a_byte_of_a_row(dtype, p, rows, hidden, group):
    n = Norm(dtype, p, rows, hidden, group)
    outs = n.q + n.scales + [n.res_out]
    before = [a.t[-1].clone() for a in outs]
    with n.comm as h:
        ccl.ccl_comm_set_debug(h, 0, 2)
        n.call(h)
        with pytest.raises(ccl.CclError) as e:
            ccl.ccl_comm_check(h)
        said = re.search(r"site (\d+), block (\d+), index (\d+)", str(e.value))
        assert e.value.status == ccl.CCL_ERR_BOUNDS and int(said[1]) == 7
        assert int(said[3]) < hidden * n.res.t.element_size()
        for a, old in zip(outs, before):
            assert torch.equal(bits(a.t[-1]), bits(old))
        got = [a.t[:-1].clone() for a in outs]
        ccl.ccl_comm_set_debug(h, 0, 0)
        n.call(h)
        torch.cuda.synchronize()
        for a, x in zip(outs, got):
            assert torch.equal(bits(a.t[:-1]), bits(x))
    n.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_with_an_infinite_reciprocal(dtype):
    """eps 0: the kernel that settles such rows' scales leaves the last row alone too."""
    n = Norm(dtype, 3, 40, 300, 0, eps=0.0)
    for a in n.x:
        a.t.zero_()
    n.res.t.fill_(1e-30)
    n.before = n.res.t.clone()
    with n.comm as h:
        for a in n.scales:
            a.t[-1] = -float("inf")
        ccl.ccl_comm_set_debug(h, 0, 2)
        n.call(h)
        with pytest.raises(ccl.CclError) as e:
            ccl.ccl_comm_check(h)
        assert e.value.status == ccl.CCL_ERR_BOUNDS
        for a in n.scales:
            assert bool((a.t[:-1] == float("inf")).all()) and float(a.t[-1]) == -float("inf")
        ccl.ccl_comm_set_debug(h, 0, 0)
        n.call(h)
    assert all(bool((a.t == float("inf")).all()) for a in n.scales)

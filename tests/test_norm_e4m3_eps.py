"""ccl_allreduce_residual_rmsnorm_e4m3 with eps 0 on rows whose mean square vanishes in fp32: 1/sqrt is infinite, so a
product h gamma of 0 has o = NaN and any other has o infinite.  A group with a NaN has scale NaN, one with
infinities alone has scale infinity, and every code is NaN (infinity times 1/infinity)."""
import pytest
import torch

from test_norm_e4m3 import Norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


TINY, SMALL = 1e-30, 4e-23          # squares of 0, and of 2^-149, which a mean over three columns or more loses


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("p, rows, hidden", [(1, 8, 64), (1, 8, 61), (2, 8, 8192), (3, 8, 5001), (8, 200, 2048), (2, 400, 512), (4, 400, 8200),
                                             (3, 400, 1001), (5, 400, 33000), (1, 400, 3)])
@pytest.mark.parametrize("zero_gamma", [False, True])
def test_means_that_vanish(dtype, group, p, rows, hidden, zero_gamma):
    n = Norm(dtype, p, rows, hidden, group, eps=0.0)
    for a in n.x:
        a.t.zero_()
    h = n.res.t
    h.fill_(TINY)
    kind = torch.arange(rows, device="cuda") % 8
    at = hidden - 1                                   # the zero of kind 1: in the last CTA's part of the row
    h[kind == 1, at] = 0.0
    h[kind == 2] = 1.0
    h[kind == 3] = 0.0
    h[kind == 4, 0] = SMALL
    h[kind == 5, 0] = SMALL
    h[kind == 5, hidden // 2] = -0.0
    h[kind == 6, 1] = float("nan")
    h[kind == 7] = -TINY
    if zero_gamma:
        n.gamma.t[hidden // 3] = 0.0
    n.before = h.clone()
    with n.comm as c:
        n.call(c)
    groups, width = n.groups, group or hidden
    nan = torch.zeros(rows, groups, dtype=torch.bool, device="cuda")
    nan[kind == 1, at // width] = True
    nan[kind == 3] = True
    nan[kind == 5, hidden // 2 // width] = True
    nan[kind == 6] = True
    if zero_gamma:
        nan[:, hidden // 3 // width] = True
    nan[kind == 2] = False
    inf = ~nan
    inf[kind == 2] = False
    s = n.scales[0].t
    assert torch.equal(torch.isnan(s), nan) and torch.equal(torch.isinf(s), inf)
    q = n.q[0].t.view(torch.float8_e4m3fn).float()
    ordinary = kind == 2
    assert bool(torch.isnan(q[~ordinary]).all()) and bool(torch.isfinite(q[ordinary]).all())
    assert torch.equal(n.res_out.t.view(torch.uint8)[kind != 6], n.merged().view(torch.uint8)[kind != 6])      # (0 + -0 is 0)
    for a, b in zip(n.scales[1:] + n.q[1:], [n.scales[0]] * (p - 1) + [n.q[0]] * (p - 1)):
        assert torch.equal(a.t.view(torch.uint8), b.t.view(torch.uint8))

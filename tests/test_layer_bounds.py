"""The checked build's tests of the accesses that the operators around layers
make (include/ccl.h, ccl_bounds_checked).  The debug hook has the checks take
buffers and lists for one row, and tensors for one element, shorter than the
call says: the last row's accesses are then recorded and not made, and the
others come out as ever.  These tests run only against the checked library
(test_zy_checked_layers.py runs them against it)."""
import os

import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import Comm, ptrs, stream
from test_expert_rows import Layer
from test_expert_sort import Choices, random_ids
from test_grads import Grads
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


def violated(h, call, site):
    ccl.ccl_comm_set_debug(h, 0, 2)
    call()
    with pytest.raises(ccl.CclError) as e:
        ccl.ccl_comm_check(h)
    assert e.value.status == ccl.CCL_ERR_BOUNDS and f"site {site}" in str(e.value)
    ccl.ccl_comm_set_debug(h, 0, 0)


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p, rows, hidden, group", [(2, 3, 512, 0), (8, 2, 8192, 128), (4, 200, 264, 32), (3, 400, 1001, 64), (1, 500, 2048, 0)])
def test_norm(dtype, p, rows, hidden, group):
    n = Norm(dtype, p, rows, hidden, group)
    outs = n.q + n.scales + [n.res_out]
    before = [a.t[-1].clone() for a in outs]
    with n.comm as h:
        violated(h, lambda: n.call(h), 7)
        for a, old in zip(outs, before):
            assert torch.equal(bits(a.t[-1]), bits(old))
        got = [a.t[:-1].clone() for a in outs]
        n.call(h)
        torch.cuda.synchronize()
        for a, x in zip(outs, got):
            assert torch.equal(bits(a.t[:-1]), bits(x))
    n.check()


@pytest.mark.parametrize("p, rows, k", [(2, 9, 2), (3, 2000, 4), (1, 9000, 3)])
@pytest.mark.parametrize("padded", [False, True])
def test_sort(p, rows, k, padded):
    valid = np.ones((p, rows), dtype=np.uint8) if padded else None
    c = Choices(random_ids(p, rows, k, 20), valid, 20, 1 << 20)
    with c.comm as h:
        for s in c.slots:
            s.t.fill_(77)
        violated(h, lambda: c.call(h), 12)
        assert all(bool((s.t[-1] == 77).all()) for s in c.slots)
        full = c.ids
        c.ids = full.copy()
        c.ids[:, -1] = -1                    # what is left: the rows before the last
        got = [s.t.clone() for s in c.slots]
        for s in c.slots:
            s.t[-1] = -1
        c.check()
        c.ids = full
        for s, x in zip(c.slots, got):
            s.t.copy_(x)
        c.call(h)
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p, rows, hidden, k", [(2, 5, 512, 2), (1, 4, 1001, 8), (3, 300, 264, 3), (2, 3, 7168, 40)])
def test_rows(dtype, p, rows, hidden, k):
    layer = Layer(dtype, p, rows, hidden, k)
    slot = layer.slot
    last = torch.zeros(p * rows, dtype=torch.bool, device="cuda")
    last[rows - 1::rows] = True

    def without_last():
        layer.slot = torch.where(last[:, None], -1, slot)

    with layer.there as h:
        violated(h, lambda: layer.dispatch(h), 11)
        without_last()
        layer.check_rows()
    layer.slot = slot
    with layer.back as h:
        old = [a.t[-1].clone() for a in layer.to_tokens]
        violated(h, lambda: layer.combine(h), 11)
        for a, x in zip(layer.to_tokens, old):
            assert torch.equal(bits(a.t[-1]), bits(x))
        layer.combine(h)
    layer.check_tokens()
    for a, x in zip(layer.to_expert, layer.before):
        a.t.copy_(x)
    with Comm(layer.tokens, layer.to_expert) as h:
        for a in layer.dweights:
            a.t.fill_(5.0)
        violated(h, lambda: layer.grad(h), 11)
        without_last()
        layer.check_rows()
        assert all(bool((a.t[-1] == 5.0).all()) for a in layer.dweights)
        for a in layer.dweights:
            a.t[-1] = 0.0
        layer.check_weights()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 8, 4096, 100003])
@pytest.mark.parametrize("offset", [0, 1])
def test_grads(dtype, n, offset):
    g = Grads([(n, dtype, 0), (n, dtype, 0)], offset=offset)
    with g.comm as h:
        violated(h, lambda: ccl.ccl_grad_norm(h, g.tensors(), g.norm.ptr(), stream()), 13)
        before = [a.t[-1].clone() for a in g.outs]
        ccl.ccl_grad_norm(h, g.tensors(), g.norm.ptr(), stream())
        violated(h, lambda: ccl.ccl_grad_clip(h, g.tensors(), 0.5, g.norm.ptr(), stream()), 13)
        for a, x in zip(g.outs, before):
            assert torch.equal(bits(a.t[-1:]), bits(x[None]))
        ins = [a.t.clone() for a in g.ins]
        g.call(h, 0.5)
    g.check(0.5, ins)

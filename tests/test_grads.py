"""ccl_grad_norm and ccl_grad_clip against their formulas in 64 bits.

Tolerances.  The norm: a thread squares and adds 32 values (fp32: 16) in four
chains of at most 8 fused multiply-adds, joined by two additions: at most 10
roundings (U32 each).  Their sum goes on as two fp32 numbers or in fp64, where
less than one U32 is lost; the root halves it, and the norm is rounded once
more: 7 U32, of which 9 are asked.  A clipped value
is its product with the factor, rounded to fp32 and to the type; the factor is
checked by itself (a sum and a quotient: 2 U32)."""
import math

import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import FLOOR, HALF_STEP, TORCH, U32, Array, Comm, assert_within, stream
from logit_testutil import rng

pytestmark = pytest.mark.gpu

CODE = {"f32": ccl.CCL_F32, "f16": ccl.CCL_F16, "bf16": ccl.CCL_BF16}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Grads:
    """Tensors with guards: a list of (n, dtype, copy)."""

    def __init__(self, parts, in_place=False, offset=0, out_offset=None, scale=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.parts, self.in_place = parts, in_place
        self.ins = [Array((n,), TORCH[d], offset, torch.randn(n, device="cuda", generator=g) * scale) for n, d, _ in parts]
        self.outs = self.ins if in_place else [Array((n,), TORCH[d], offset if out_offset is None else out_offset) for n, d, _ in parts]
        self.norm = Array((2,), torch.float32)
        self.buffer = Array((4,), torch.float32)
        self.comm = Comm([self.buffer])
        self.comm.arrays += self.ins + self.outs + [self.norm]

    def tensors(self):
        return [ccl.Tensor(i.ptr(), o.ptr(), n, CODE[d], c) for (n, d, c), i, o in zip(self.parts, self.ins, self.outs)]

    def exact(self):
        """The norm as a Python float (exact sums of fp64 squares where they are finite)."""
        return math.sqrt(sum(float(a.t.double().square().sum()) for a, (_, _, c) in zip(self.ins, self.parts) if not c))

    def call(self, h, max_norm):
        ccl.ccl_grad_norm(h, self.tensors(), self.norm.ptr(), stream())
        ccl.ccl_grad_clip(h, self.tensors(), max_norm, self.norm.ptr(), stream())

    def check(self, max_norm, before, norm=None):
        want = self.exact() if norm is None else norm
        got, factor = self.norm.t.tolist()
        if want >= 2.0 ** 128:          # above fp32's range: the header says infinity
            assert got == INF
        else:
            assert abs(got - want) <= 9 * U32 * want + 2.0 ** -149, (got, want)
        exact = min(1.0, max_norm / (got + float(np.float32(1e-6))))
        assert abs(factor - exact) <= 2 * U32 * exact + 2.0 ** -149
        for a, x, (n, d, _) in zip(self.outs, before, self.parts):
            want = x.double() * factor
            assert_within(a.t, want, (HALF_STEP[d] + U32 * (d != "f32")) * want.abs() + FLOOR[d], d)


def run(parts, max_norm=1.0, **layout):
    g = Grads(parts, **layout)
    before = [a.t.clone() for a in g.ins]
    norm = g.exact()
    with g.comm as h:
        g.call(h, max_norm)
    g.check(max_norm, before, norm)
    if not g.in_place:
        for a, x in zip(g.ins, before):
            assert torch.equal(a.t, x)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 255, 1000, 4095, 4096, 4097, 8191, 8192, 8193, 100003, 3000001])
@pytest.mark.parametrize("in_place", [False, True])
def test_one_tensor(dtype, n, in_place):
    run([(n, dtype, 0)], in_place=in_place)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset, out_offset", [(1, None), (3, None), (7, None), (0, 1), (5, 2), (3, 0)])
@pytest.mark.parametrize("n", [1, 5, 17, 20003])
def test_alignment(dtype, offset, out_offset, n):
    run([(n, dtype, 0)], offset=offset, out_offset=out_offset)
    if out_offset is None:
        run([(n, dtype, 0)], offset=offset, in_place=True)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 895, 896, 897, 1800])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_tensors(count, in_place):
    g = rng(count)
    sizes = np.exp(g.uniform(0, 9, count)).astype(int)
    sizes[g.random(count) < 0.1] = 0
    parts = [(int(n), str(g.choice(["f32", "f16", "bf16"])), int(g.random() < 0.1)) for n in sizes]
    run(parts, in_place=in_place, offset=int(g.integers(0, 4)))


@pytest.mark.parametrize("parts", [[(60000001, "bf16", 0), (70, "f32", 0), (9000003, "f16", 1)], [(150000000, "f32", 0), (50000003, "f32", 0), (1, "bf16", 0)]])
@pytest.mark.parametrize("in_place", [False, True])
def test_large_tensors(parts, in_place):
    """Several CTAs have a share of the tiles."""
    run(parts, in_place=in_place, offset=1)


def test_no_tensor():
    for parts in ([], [(0, "f32", 0)], [(5, "f32", 1)], [(0, "bf16", 0)] * 100):
        g = Grads(parts)
        with g.comm as h:
            ccl.ccl_grad_norm(h, g.tensors(), g.norm.ptr(), stream())
            ccl.ccl_grad_clip(h, g.tensors(), 2.0, g.norm.ptr(), stream())
        assert g.norm.t.tolist() == [0.0, 1.0]


def test_null_of_no_elements():
    norm, buffer = Array((2,), torch.float32), Array((4,), torch.float32)
    with Comm([buffer]) as h:
        ccl.ccl_grad_norm(h, [ccl.Tensor(0, 0, 0, 0, 0)], norm.ptr(), stream())
        ccl.ccl_grad_clip(h, [ccl.Tensor(0, 0, 0, 0, 0)], 1.0, norm.ptr(), stream())
    assert norm.t.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("dtype, scale", [("f32", 1e30), ("f32", 1e19), ("f32", 1e-19), ("f32", 1e-30), ("f32", 1e-42), ("bf16", 1e37),
                                          ("bf16", 1e-30), ("bf16", 1e-38), ("f16", 2e4), ("f16", 1e-7), ("f32", 1e-12), ("f32", 2e-13)])
@pytest.mark.parametrize("n", [1, 100, 50001])
def test_scales(dtype, scale, n):
    """Values whose squares leave fp32's range, alone and beside ordinary ones."""
    run([(n, dtype, 0)], scale=scale, max_norm=1e-3)
    run([(n, dtype, 0), (10000, "bf16", 0)], scale=scale, max_norm=3.0)


def test_mixed_scales():
    """Large and small values in one group, one tile and one tensor."""
    g = Grads([(30000, "f32", 0), (30000, "bf16", 0)])
    for a in g.ins:
        a.t.mul_(10.0 ** torch.linspace(-37, 36, 30000, device="cuda")[torch.randperm(30000, device="cuda")].to(a.t.dtype))
    before = [a.t.clone() for a in g.ins]
    with g.comm as h:
        g.call(h, 1e30)
    g.check(1e30, before)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("values, want", [((NAN,), NAN), ((INF,), INF), ((-INF, 1.0), INF), ((INF, NAN), NAN), ((NAN, -INF), NAN)])
@pytest.mark.parametrize("at", [0, 70001])
def test_not_finite(dtype, values, want, at):
    """A NaN makes every gradient NaN; an infinity makes the factor 0, and itself NaN."""
    g = Grads([(80000, dtype, 0), (100, "f32", 0)])
    for i, v in enumerate(values):
        g.ins[0].t[at + 100 * i] = v
    with g.comm as h:
        g.call(h, 1.0)
    got, factor = g.norm.t.tolist()
    if math.isnan(want):
        assert math.isnan(got) and math.isnan(factor)
        assert all(bool(torch.isnan(a.t).all()) for a in g.outs)
    else:
        assert got == INF and factor == 0.0
        for a, o in zip(g.ins, g.outs):
            assert torch.equal(torch.isnan(o.t), torch.isinf(a.t)) and bool((o.t[torch.isfinite(a.t)] == 0).all())


def test_a_norm_above_the_range():
    g = Grads([(64, "f32", 0)])
    g.ins[0].t.fill_(3e38)
    with g.comm as h:
        ccl.ccl_grad_norm(h, g.tensors(), g.norm.ptr(), stream())
    assert float(g.norm.t[0]) == INF


def test_a_copy_is_clipped_and_not_counted():
    g = Grads([(1000, "bf16", 0), (1000, "bf16", 1), (3, "f32", 7)])
    g.ins[2].t.fill_(NAN)
    norm = math.sqrt(float(g.ins[0].t.double().square().sum()))
    with g.comm as h:
        g.call(h, 1.0)
    assert abs(float(g.norm.t[0]) - norm) <= 9 * U32 * norm
    factor = float(g.norm.t[1])
    want = g.ins[1].t.double() * factor
    assert_within(g.outs[1].t, want, (HALF_STEP["bf16"] + U32) * want.abs())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_below_the_limit(dtype):
    """Nothing changes, in place or not, down to a signed zero."""
    for in_place in (False, True):
        g = Grads([(5003, dtype, 0)], in_place=in_place, offset=1)
        g.ins[0].t[::7] = -0.0
        before = g.ins[0].t.clone()
        with g.comm as h:
            g.call(h, 1e4)
        assert float(g.norm.t[1]) == 1.0
        assert torch.equal(g.outs[0].t.view(torch.uint8), before.view(torch.uint8))


def test_a_limit_of_zero():
    g = Grads([(5003, "f32", 0)])
    with g.comm as h:
        g.call(h, 0.0)
    assert float(g.norm.t[1]) == 0.0 and not bool(g.outs[0].t.any())


def test_another_norm():
    """clip takes the norm that it is given."""
    g = Grads([(5003, "f32", 0)])
    g.norm.t.copy_(torch.tensor([8.0, -1.0]))
    with g.comm as h:
        ccl.ccl_grad_clip(h, g.tensors(), 2.0, g.norm.ptr(), stream())
    factor = float(g.norm.t[1])
    assert float(g.norm.t[0]) == 8.0 and abs(factor - 0.25) < 1e-6
    assert torch.equal(g.outs[0].t, g.ins[0].t * factor)


def test_zeros_of_either_sign():
    for dtype in ("f32", "bf16"):
        g = Grads([(9000, dtype, 0), (5, dtype, 0)])
        g.ins[0].t.fill_(-0.0)
        g.ins[1].t.fill_(0.0)
        with g.comm as h:
            g.call(h, 1.0)
        assert g.norm.t.tolist() == [0.0, 1.0]
        assert torch.equal(g.outs[0].t.view(torch.uint8), g.ins[0].t.view(torch.uint8))


def test_the_last_launch_is_described():
    """An operator's words, then a collective's, from one communicator."""
    g = Grads([(100, "f32", 0)] * 2)
    with g.comm as h:
        ccl.ccl_grad_norm(h, g.tensors(), g.norm.ptr(), stream())
        assert ccl.ccl_comm_last_launch(h).startswith("grad_norm ") and "kernels=1" in ccl.ccl_comm_last_launch(h)
        ccl.ccl_allreduce(h, "sum", "f32", 4, "ring", stream())
        assert ccl.ccl_comm_last_launch(h).startswith("allreduce")
        before = ccl.ccl_comm_launch_count(h)
        ccl.ccl_grad_clip(h, g.tensors(), 1.0, g.norm.ptr(), stream())
        assert ccl.ccl_comm_last_launch(h).startswith("grad_clip ") and ccl.ccl_comm_launch_count(h) == before + 1


def test_the_same_bits():
    a, b = Grads([(3000001, "bf16", 0), (70000, "f32", 0)]), Grads([(3000001, "bf16", 0), (70000, "f32", 0)])
    for g in (a, b):
        with g.comm as h:
            g.call(h, 1.0)
    assert torch.equal(a.norm.t, b.norm.t) and all(torch.equal(x.t, y.t) for x, y in zip(a.outs, b.outs))


def test_graphs_that_share_a_communicator():
    a, b = Grads([(100003, "bf16", 0)] * 70), Grads([(5, "f32", 0), (999, "f16", 0)], in_place=True)
    with a.comm as h:
        a.call(h, 1.0)
        b.call(h, 1.0)
        torch.cuda.synchronize()
        graphs = []
        for g in (a, b):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                g.call(h, 1.0)
        for scale in (2.0, 0.5):
            before = []
            for g in (a, b):
                for x in g.ins:
                    x.t.mul_(scale * 3)
                before.append([x.t.clone() for x in g.ins])
            norms = [a.exact(), b.exact()]
            graphs[0].replay()
            graphs[1].replay()
            torch.cuda.synchronize()
            for g, x, n in zip((a, b), before, norms):
                g.check(1.0, x, n)
    with b.comm:
        pass


def test_another_stream():
    g = Grads([(70000, "bf16", 0)])
    before = [a.t.clone() for a in g.ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with g.comm as h, torch.cuda.stream(side):
        g.call(h, 1.0)
    g.check(1.0, before)


def test_beyond_32_bits():
    """A tensor of more than 2^32 elements: its last values count and are clipped."""
    n = (1 << 32) + 70003
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[-3:] = 2.0
    x[1 << 32] = 1.0
    norm, buffer = Array((2,), torch.float32), Array((4,), torch.float32)
    with Comm([buffer]) as h:
        t = (ccl.Tensor * 1)(ccl.Tensor(x.data_ptr(), x.data_ptr(), n, ccl.CCL_BF16, 0))
        ccl.ccl_grad_norm(h, t, norm.ptr(), stream())
        ccl.ccl_grad_clip(h, t, 1.0, norm.ptr(), stream())
    want = math.sqrt(13.0)
    got, factor = norm.t.tolist()
    assert abs(got - want) <= 9 * U32 * want
    assert x[-3:].tolist() == [float(torch.tensor(2 * factor).bfloat16())] * 3
    assert float(x[1 << 32]) == float(torch.tensor(factor).bfloat16()) and int(torch.count_nonzero(x)) == 4

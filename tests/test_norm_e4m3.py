"""ccl_allreduce_residual_rmsnorm_e4m3 against its formula in 64 bits.

Tolerances.  The merged residual is exact: the same fp32 sums in the schedule's
order and the same roundings.  The sum of squares is an fp32 sum of positive
terms: a thread adds at most hidden / 128 + 8 of them in a row and at most 5 +
32 + 8 additions join the threads, each U32; 1 / sqrt halves that and adds a
quotient, a sum, a root and a quotient; o has two more products, a scale one
quotient: (hidden / 128 + 53) / 2 + 7 in all, in U32.  A code is off by at
most half a step of e4m3, 2^-4 of its value or 2^-10, beside what o and the
scale are off."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import TORCH, U32, Array, Comm, assert_within, ptrs, stream
from logit_testutil import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Norm:
    def __init__(self, dtype, p, rows, hidden, group=0, offset=0, out_offset=None, in_place=False, schedule="ring", eps=1e-6, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 13 * rows + hidden)
        T = TORCH[dtype]
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.args = (dtype, p, rows, hidden, group)
        self.schedule, self.eps = schedule, eps
        self.x = [Array((rows, hidden), T, offset, rand(rows, hidden)) for _ in range(p)]
        self.q = [Array((rows, hidden), torch.uint8, offset if out_offset is None else out_offset) for _ in range(p)]
        self.groups = -(-hidden // group) if group else 1
        self.scales = [Array((rows, self.groups), torch.float32, offset) for _ in range(p)]
        self.res = Array((rows, hidden), T, offset, rand(rows, hidden) * 2)
        self.res_out = self.res if in_place else Array((rows, hidden), T, offset)
        self.gamma = Array((hidden,), T, offset, 1 + 0.3 * rand(hidden))
        self.before = self.res.t.clone()
        self.comm = Comm(self.x, self.q)
        self.comm.arrays += self.scales + [self.res, self.res_out, self.gamma]

    def call(self, h):
        dtype, p, rows, hidden, group = self.args
        ccl.ccl_allreduce_residual_rmsnorm_e4m3(h, dtype, rows, hidden, self.res.ptr(), self.res_out.ptr(), self.gamma.ptr(),
                                                ptrs(self.scales), group, self.eps, self.schedule, stream())

    def merged(self):
        """h, from fp32 sums in the schedule's order."""
        dtype, p, rows, hidden, _ = self.args
        bounds, order = ccl.ccl_schedule_build(p, rows * hidden, self.schedule)
        x = [a.t.reshape(-1).float() for a in self.x]
        y = torch.empty_like(x[0])
        for c in range(p):
            part = slice(bounds[c], bounds[c + 1])
            acc = x[order[c][0]][part].clone()
            for r in order[c][1:]:
                acc += x[r][part]
            y[part] = acc
        T = TORCH[dtype]
        return (y.to(T).float() + self.before.reshape(-1).float()).to(T).view(rows, hidden)

    def check(self):
        dtype, p, rows, hidden, group = self.args
        h = self.merged()
        assert torch.equal(self.res_out.t.view(torch.uint8), h.view(torch.uint8))
        h = h.double()
        o = h * self.gamma.t.double() / (h.square().mean(1, keepdim=True) + float(np.float32(self.eps))).sqrt()
        width = group or hidden
        pad = torch.nn.functional.pad(o, (0, self.groups * width - hidden)).view(rows, self.groups, width)
        scale = (pad.abs().amax(2) / 448).clamp(min=2.0 ** -126)
        tol = ((hidden / 128 + 53) / 2 + 7) * U32
        got = self.scales[0].t
        assert_within(got, scale, tol * scale, "scales")
        per = got.double().repeat_interleave(width, 1)[:, :hidden]
        v = o / per
        q = self.q[0].t.view(torch.float8_e4m3fn).float()
        assert_within(q, v, torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + 2 * tol * v.abs(), "codes")
        for a in self.q[1:]:
            assert torch.equal(a.t, self.q[0].t)
        for a in self.scales[1:]:
            assert torch.equal(a.t, got)


def run(*args, **more):
    n = Norm(*args, **more)
    with n.comm as h:
        n.call(h)
    n.check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("p, rows, hidden", [
    (1, 1, 8), (1, 1, 1), (2, 3, 128), (8, 1, 8192), (8, 16, 7168), (4, 40, 4096), (3, 7, 1000), (2, 160, 512), (4, 200, 8200),
    (8, 310, 1536), (1, 400, 2048), (2, 333, 257), (3, 320, 8192), (64, 2, 256), (13, 5, 129), (1, 2, 40000), (1, 700, 16384), (2, 310, 33000)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_sizes(dtype, p, rows, hidden, group):
    run(dtype, p, rows, hidden, group)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("offset, out_offset", [(1, None), (4, None), (8, None), (0, 4), (0, 3), (8, 16)])
def test_alignment(dtype, group, offset, out_offset):
    run(dtype, 2, 5, 520, group, offset=offset, out_offset=out_offset)
    run(dtype, 4, 500, 264, group, offset=offset, out_offset=out_offset)


@pytest.mark.parametrize("rows", [2, 200, 500])
@pytest.mark.parametrize("schedule", ["ring", "allpairs"])
def test_in_place_residual_and_schedules(rows, schedule):
    run("bf16", 4, rows, 1024, 128, in_place=True, schedule=schedule)
    run("f16", 3, rows, 1025, 32, in_place=True, schedule=schedule)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p, rows, hidden", [(3, 1, 8), (3, 1, 40), (8, 3, 6104), (3, 7, 2056), (4, 401, 968), (8, 1, 24), (7, 500, 264), (64, 5, 72)])
@pytest.mark.parametrize("schedule", ["ring", "allpairs"])
def test_chunks_that_end_inside_a_group_of_elements(dtype, p, rows, hidden, schedule):
    """Rows of whole 16-byte groups whose chunks end anywhere: each element has its own chunk's order."""
    assert rows * hidden % p or rows * hidden // p % 8
    run(dtype, p, rows, hidden, 32, schedule=schedule)


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("rows", [3, 400])
def test_zeros_and_small_rows(group, rows):
    """A row of nothing has scale 2^-126 and codes of 0 (of -0, 0x80, where gamma is negative); eps 0 and tiny rows stay finite where 1/rms is."""
    n = Norm("f32", 2, rows, 256, group)
    for a in n.x:
        a.t.zero_()
    n.res.t[0], n.res.t[1] = 0.0, 1e-15
    n.res.t[2, 10:] = 0.0
    n.before = n.res.t.clone()
    with n.comm as h:
        n.call(h)
    n.check()
    assert bool((n.q[0].t[0].view(torch.float8_e4m3fn).float() == 0).all()) and bool((n.scales[0].t[0] == 2.0 ** -126).all())


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("rows", [4, 400])
def test_not_finite(group, rows):
    """A NaN in a row: every scale and code of the row is NaN.  A NaN or an infinity of gamma: that of its column's groups."""
    n = Norm("bf16", 2, rows, 512, group)
    n.x[1].t[1, 100] = float("nan")
    with n.comm as h:
        n.call(h)
        torch.cuda.synchronize()
        q = n.q[0].t.view(torch.float8_e4m3fn).float()
        bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
        bad[1] = True
        assert torch.equal(torch.isnan(n.scales[0].t).all(1), bad) and torch.equal(torch.isnan(n.scales[0].t).any(1), bad)
        assert torch.equal(torch.isnan(q).all(1), bad) and torch.equal(torch.isnan(q).any(1), bad)
        n.x[1].t[1, 100] = 1.0
        n.gamma.t[70] = float("inf")
        n.call(h)
        torch.cuda.synchronize()
        q, s = n.q[0].t.view(torch.float8_e4m3fn).float(), n.scales[0].t
        zero = n.merged()[:, 70] == 0                     # 0 times infinity is NaN
        assert int(zero.sum()) < rows / 2
        hit = torch.tensor([True] if not group else [False, True] + [False] * 6, device="cuda")
        assert torch.equal(torch.isinf(s), hit[None] & ~zero[:, None]) and torch.equal(torch.isnan(s), hit[None] & zero[:, None])
        of = slice(64, 128) if group else slice(0, 512)
        assert bool(torch.isnan(q[:, 70]).all()) and bool(torch.isnan(q[zero, of]).all())
        assert int((q[~zero, of] == 0).sum()) == int((~zero).sum()) * (of.stop - of.start - 1)


def test_codes_at_the_edges():
    """Values that are codes come out as themselves, and values between them round to even."""
    codes = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()     # 0 ... 448
    mid = (codes[1:] + codes[:-1]) / 2
    row = torch.cat([codes, mid, -codes[1:]])
    hidden = row.numel()
    n = Norm("f32", 1, 1, hidden, 0, eps=0.0)
    # gamma carries the values: h is 1 everywhere, so 1/rms is 1 and o is gamma
    n.x[0].t.fill_(0.25)
    n.res.t.fill_(0.75)
    n.gamma.t.copy_(row)
    with n.comm as h:
        n.call(h)
    assert float(n.scales[0].t) == 1.0
    want = row.to(torch.float8_e4m3fn)
    assert torch.equal(n.q[0].t[0].view(torch.float8_e4m3fn).float(), want.float())


@pytest.mark.parametrize("rows", [2, 200, 1000])
def test_captured(rows):
    n = Norm("bf16", 4, rows, 2048, 128)
    with n.comm as h:
        n.call(h)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            n.call(h)
        for i in (1, 2):
            n.x[0].t.mul_(1.5)
            graph.replay()
            torch.cuda.synchronize()
            n.check()


def test_the_exchange_gives_up():
    """A withheld sum: the bounded wait runs out, the call reports it, and the next call is right."""
    n = Norm("bf16", 8, 2, 8192, 0)
    h = n.comm.h
    ccl.ccl_comm_set_debug(h, 20_000_000, 1)
    n.call(h)
    with pytest.raises(ccl.CclError) as e:
        ccl.ccl_comm_check(h)
    assert e.value.status == ccl.CCL_ERR_TIMEOUT
    ccl.ccl_comm_set_debug(h, 0, 0)
    with n.comm:
        n.call(h)
    n.check()


def test_beyond_32_bits():
    rows, hidden = 65600, 65536
    x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros_like(x)
    q = torch.zeros(rows, hidden, dtype=torch.uint8, device="cuda")
    gamma = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    scales = torch.zeros(rows, hidden // 128, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x[-2:] = torch.randn(2, hidden, device="cuda", generator=g).bfloat16()
    h = ccl.ccl_comm_create(1, [x.data_ptr()])
    ccl.ccl_comm_set_outputs(h, [q.data_ptr()])
    ccl.ccl_allreduce_residual_rmsnorm_e4m3(h, "bf16", rows, hidden, res.data_ptr(), res.data_ptr(), gamma.data_ptr(),
                                            [scales.data_ptr()], 128, 1e-6, "ring", stream())
    ccl.ccl_comm_check(h)
    ccl.ccl_comm_destroy(h)
    assert torch.equal(res[-2:], x[-2:]) and not bool(q[:-2].any())
    o = x[-2:].double() / (x[-2:].double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    tol = ((hidden / 128 + 53) / 2 + 7) * U32
    scale = o.view(2, -1, 128).abs().amax(2) / 448
    assert_within(scales[-2:], scale, tol * scale)
    v = o / scales[-2:].double().repeat_interleave(128, 1)
    assert_within(q[-2:].view(torch.float8_e4m3fn).float(), v,
                  torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + 2 * tol * v.abs())


@pytest.mark.parametrize("seed", range(20))
def test_random(seed):
    g = rng(900 + seed)
    rows, hidden = int(np.exp(g.uniform(0, 7))), int(np.exp(g.uniform(3, 9.5)))
    if g.random() < 0.6:
        hidden = -(-hidden // 8) * 8
    run(str(g.choice(["f32", "f16", "bf16"])), int(g.choice([1, 2, 3, 4, 8])), rows, hidden, int(g.choice([0, 32, 64, 128])),
        schedule=str(g.choice(["ring", "allpairs"])), in_place=bool(g.random() < 0.3), seed=seed)

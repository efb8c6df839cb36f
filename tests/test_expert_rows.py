"""ccl_expert_dispatch, ccl_expert_combine and ccl_expert_combine_grad against
their formulas in 64 bits.

Tolerances.  A product is rounded to fp32 (U32 of it) and then to the type (half
a step).  combine adds k products with k fused multiply-adds, each rounded: k
U32 of the sum of the products' sizes.  A weight's gradient is a sum over the
hidden columns in fp32: a thread adds at most hidden / 32 + 8 products in a
row (a warp or more shares a row, 8 columns at a time), then at most 15 more
additions join the threads; of a narrow row, which 8 or 16 threads share, a
thread adds at most 12 (8 columns, and 4 of the edges'), and 4 more join them."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import FLOOR, HALF_STEP, TORCH, U32, Array, Comm, assert_within, ptrs, sort_by_expert, stream
from logit_testutil import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    """Slots of random choices, and everything the three operators read and write."""

    def __init__(self, dtype, p, rows, hidden, k, capacity=None, offset=0, weighted=True, seed=0, experts=None, slots=None):
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * rows + hidden)
        self.dtype, self.p, self.rows, self.hidden, self.k = dtype, p, rows, hidden, k
        self.capacity = capacity = (rows * k * p if capacity is None else capacity)
        experts = experts or 2 * p + 1
        if slots is None:
            ids = rng(seed + rows).integers(-1, experts, (p, rows, k)).astype(np.int32)
            slots = sort_by_expert(ids, None, experts, capacity)[0]
        self.slot = torch.from_numpy(slots).cuda().long().view(p * rows, k)
        T = TORCH[dtype]
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.tokens = [Array((rows, hidden), T, offset, rand(rows, hidden)) for _ in range(p)]
        self.expert = [Array((capacity, hidden), T, offset, rand(capacity, hidden)) for _ in range(p)]
        self.slots = [Array((rows, k), torch.int32, offset, torch.from_numpy(s)) for s in slots]
        self.weights = [Array((rows, k), torch.float32, offset, rand(rows, k)) for _ in range(p)] if weighted else None
        self.dweights = [Array((rows, k), torch.float32, offset) for _ in range(p)]
        self.to_tokens = [Array((rows, hidden), T, offset) for _ in range(p)]
        self.to_expert = [Array((capacity, hidden), T, offset) for _ in range(p)]
        self.before = [a.t.clone() for a in self.to_expert]
        self.there = Comm(self.tokens, self.to_expert)
        self.back = Comm(self.expert, self.to_tokens)
        self.there.arrays += self.slots + self.dweights + self.expert

    def dispatch(self, h):
        ccl.ccl_expert_dispatch(h, self.dtype, self.rows, self.hidden, self.k, ptrs(self.slots), ptrs(self.weights),
                                self.capacity, stream())

    def combine(self, h):
        ccl.ccl_expert_combine(h, self.dtype, self.rows, self.hidden, self.k, ptrs(self.slots), ptrs(self.weights),
                               self.capacity, stream())

    def grad(self, h):
        ccl.ccl_expert_combine_grad(h, self.dtype, self.rows, self.hidden, self.k, ptrs(self.slots), ptrs(self.weights),
                                    ptrs(self.expert), self.capacity, ptrs(self.dweights), stream())

    def w(self):
        if self.weights is None:
            return torch.ones(self.p * self.rows, self.k, dtype=torch.float64, device="cuda")
        return torch.cat([a.t for a in self.weights]).double()

    def pairs(self):
        """(token, choice, row of all ranks' buffers) of the choices with a row."""
        at = torch.nonzero((self.slot >= 0) & (self.slot < self.p * self.capacity))
        return at[:, 0], at[:, 1], self.slot[at[:, 0], at[:, 1]]

    def check_rows(self):
        """The experts' rows that dispatch and the gradient write, and that others are as they were."""
        token, choice, row = self.pairs()
        got, old = (torch.cat(list(x)) for x in ((a.t for a in self.to_expert), self.before))
        kept = torch.ones(len(got), dtype=torch.bool, device="cuda")
        kept[row] = False
        assert torch.equal(got[kept].view(torch.uint8), old[kept].view(torch.uint8))
        x = torch.cat([a.t for a in self.tokens])[token]
        if self.weights is None:
            assert torch.equal(got[row].view(torch.uint8), x.view(torch.uint8))
            return
        want = x.double() * self.w()[token, choice][:, None]
        assert_within(got[row], want, (HALF_STEP[self.dtype] + 2 * U32) * want.abs() + FLOOR[self.dtype], "rows")

    def check_tokens(self):
        token, choice, row = self.pairs()
        z = torch.cat([a.t for a in self.expert])
        want = torch.zeros(self.p * self.rows, self.hidden, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        w = self.w()
        for j in range(self.k):
            of = choice == j
            part = z[row[of]].double() * w[token[of], j][:, None]
            want.index_add_(0, token[of], part)
            size.index_add_(0, token[of], part.abs())
        tol = HALF_STEP[self.dtype] * want.abs() + 2 * self.k * U32 * size + FLOOR[self.dtype]
        assert_within(torch.cat([a.t for a in self.to_tokens]), want, tol, "tokens")

    def check_weights(self):
        token, choice, row = self.pairs()
        z, x = torch.cat([a.t for a in self.expert]), torch.cat([a.t for a in self.tokens])
        want = torch.zeros(self.p * self.rows, self.k, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for j in range(self.k):
            of = choice == j
            part = z[row[of]].double() * x[token[of]].double()
            want[token[of], j] = part.sum(1)
            size[token[of], j] = part.abs().sum(1)
        tol = (self.hidden / 32 + 8 + 15) * U32 * size + FLOOR["f32"]
        assert_within(torch.cat([a.t for a in self.dweights]), want, tol, "dweights")

    def all(self):
        with self.there as h:
            self.dispatch(h)
        self.check_rows()
        with self.back as h:
            self.combine(h)
        self.check_tokens()
        for a, old in zip(self.to_expert, self.before):
            a.t.copy_(old)
        with Comm(self.tokens, self.to_expert) as h:
            self.grad(h)
        assert all(a.guarded() for a in self.dweights)
        self.check_rows()
        self.check_weights()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("p, rows, hidden, k", [
    (1, 1, 8, 1), (1, 1, 1, 1), (1, 3, 7168, 8), (2, 5, 4096, 2), (8, 16, 1536, 8), (3, 17, 1001, 3), (4, 33, 130, 6), (2, 1, 3, 5),
    (8, 2, 8200, 1), (1, 40, 264, 9), (2, 7, 515, 17), (64, 2, 96, 4), (1, 300, 2048, 4), (2, 3, 40, 200)])
@pytest.mark.parametrize("weighted", [False, True])
def test_sizes(dtype, p, rows, hidden, k, weighted):
    Layer(dtype, p, rows, hidden, k, weighted=weighted).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [256, 260, 257, 258])
@pytest.mark.parametrize("offset", [1, 2, 4, 8])
def test_alignment(dtype, hidden, offset):
    Layer(dtype, 2, 9, hidden, 3, offset=offset).all()


@pytest.mark.parametrize("capacity", [0, 1, 10, 40])
def test_full_buffers(capacity):
    """Choices without a row: nothing is written for them, their part of the sum and their weight's gradient are 0."""
    Layer("bf16", 3, 20, 520, 4, capacity=capacity).all()


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, 120])
def test_values_that_are_no_slot(bad):
    slots = np.full((2, 15, 4), bad, dtype=np.int32)
    Layer("f32", 2, 15, 72, 4, capacity=60, slots=slots).all()
    slots[0, ::2, 1] = np.arange(8) * 7
    slots[1, 3, :] = [119, bad, 60, 59]
    Layer("f16", 2, 15, 72, 4, capacity=60, slots=slots).all()


def test_one_row_for_many_tokens():
    """combine may read a row more than once."""
    layer = Layer("bf16", 2, 30, 136, 4, capacity=5, slots=rng(0).integers(-1, 10, (2, 30, 4)).astype(np.int32))
    with layer.back as h:
        layer.combine(h)
    layer.check_tokens()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hidden", [64, 61])
def test_not_finite(dtype, hidden):
    """Infinities and NaN travel with their own rows and no others; rows that no choice has are not read."""
    layer = Layer(dtype, 2, 12, hidden, 3, capacity=50)
    token, choice, row = layer.pairs()
    z = torch.full((2 * 50, hidden), float("nan"), device="cuda", dtype=TORCH[dtype])
    z[row] = torch.cat([a.t for a in layer.expert])[row]
    z[row[0]], z[row[5], 3], z[row[9], 1] = float("inf"), float("nan"), -float("inf")
    for a, part in zip(layer.expert, z.split(50)):
        a.t.copy_(part)
    layer.tokens[1].t[4, 2] = float("nan")
    layer.tokens[0].t[5, 7] = float("inf")
    layer.all()


def test_bits_are_copied():
    """Without weights every bit pattern arrives, and int32 rows too."""
    layer = Layer("f16", 2, 64, 256, 2, weighted=False)
    for a in layer.tokens:
        a.t.view(torch.int16).copy_(torch.randint(-2 ** 15, 2 ** 15, a.t.shape, device="cuda", dtype=torch.int16))
    with layer.there as h:
        layer.dispatch(h)
    layer.check_rows()
    for a, old in zip(layer.to_expert, layer.before):
        a.t.copy_(old)
    with Comm(layer.tokens, layer.to_expert) as h:
        ccl.ccl_expert_dispatch(h, "i32", 64, 128, 2, ptrs(layer.slots), None, layer.capacity, stream())
    layer.check_rows()


@pytest.mark.parametrize("hidden, offset", [(33, 0), (64, 1), (2, 0), (1, 3), (1000, 2)])
def test_int32_rows_anywhere(hidden, offset):
    """Rows of 4-byte words that are no 16-byte groups: scales, or codes of an odd width."""
    layer = Layer("f32", 3, 30, hidden, 2, offset=offset, weighted=False)
    for a in layer.tokens:
        a.t.view(torch.int32).copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, a.t.shape, device="cuda"))
    with layer.there as h:
        ccl.ccl_expert_dispatch(h, "i32", 30, hidden, 2, ptrs(layer.slots), None, layer.capacity, stream())
    layer.check_rows()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, hidden, k", [
    (25000, 8, 2), (25000, 64, 3), (25000, 100, 1), (24999, 128, 8), (12001, 256, 2), (12001, 512, 1), (9001, 1024, 5), (5003, 2048, 2),
    (4001, 4096, 2), (25000, 3, 2), (25000, 31, 3), (25000, 61, 2), (20001, 129, 2), (12001, 203, 9), (9001, 301, 2), (5003, 1001, 3), (3001, 2002, 2)])
def test_many_tokens(dtype, rows, hidden, k):
    """Teams of 8 to 256 threads: few threads a token where there are many tokens; some choices without a row."""
    p, capacity = 2, rows * k
    slots = rng(hidden).permutation(p * capacity).astype(np.int32).reshape(p, rows, k)
    slots[rng(rows).random((p, rows, k)) < 0.05] = -1
    Layer(dtype, p, rows, hidden, k, capacity=capacity, slots=slots).all()


@pytest.mark.parametrize("hidden", [16, 13])
def test_thousands_of_choices(hidden):
    """Lists of choices that need more shared memory than a kernel has without asking."""
    Layer("bf16", 1, 2, hidden, 3100).all()


@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_by_differences(weighted):
    """The three operators' gradients against central differences of sum(c * y), in fp32 with inputs that are small whole
    numbers, so that everything is exact."""
    p, rows, hidden, k = 2, 5, 12, 3
    layer = Layer("f32", p, rows, hidden, k, capacity=20, weighted=weighted)
    g = rng(5)
    whole = lambda shape: torch.from_numpy(g.integers(-4, 5, shape).astype(np.float32)).cuda()
    for arrays in (layer.tokens, layer.expert, layer.weights or []):
        for a in arrays:
            a.t.copy_(whole(a.t.shape))
    dy = [a.t.clone() for a in layer.tokens]

    def value():
        with Comm(layer.expert, layer.to_tokens) as h:
            layer.combine(h)
        return float(sum((a.t * d).sum(dtype=torch.float64) for a, d in zip(layer.to_tokens, dy)))

    def slope(a, i):
        old = float(a.t.view(-1)[i])
        ends = []
        for step in (1.0, -1.0):
            a.t.view(-1)[i] = old + step
            ends.append(value())
        a.t.view(-1)[i] = old
        return (ends[0] - ends[1]) / 2

    for a in layer.to_expert:
        a.t.zero_()
    with Comm(layer.tokens, layer.to_expert) as h:
        layer.grad(h)
    for r in range(p):
        for i in range(0, layer.expert[r].t.numel(), 5):
            assert slope(layer.expert[r], i) == float(layer.to_expert[r].t.view(-1)[i])
        for i in range(rows * k if weighted else 0):
            assert slope(layer.weights[r], i) == float(layer.dweights[r].t.view(-1)[i])
    # dispatch is linear: <dispatch(x), z> = <x, combine(z)>
    with Comm(layer.tokens, layer.to_expert) as h:
        layer.dispatch(h)
    left = sum((a.t.double() * b.t.double()).sum() for a, b in zip(layer.to_expert, layer.expert))
    assert float(left) == value()


def test_rows_beyond_32_bits():
    """Elements beyond 2^32 of an expert buffer."""
    rows, hidden, capacity = 6, 65544, 70000
    slots = np.array([[[69999, 0], [65536, 65535], [-1, 32768], [12345, 69998], [65537, 1], [40000, 50000]]], dtype=np.int32)
    T = torch.bfloat16
    tokens, back = Array((rows, hidden), T, 0, torch.randn(rows, hidden, device="cuda")), Array((rows, hidden), T)
    z = torch.zeros(capacity, hidden, dtype=T, device="cuda")
    dz = torch.zeros_like(z)
    d_slots, dw = Array((rows, 2), torch.int32, 0, torch.from_numpy(slots[0])), Array((rows, 2), torch.float32)
    h = ccl.ccl_comm_create(1, [tokens.ptr()])
    ccl.ccl_comm_set_outputs(h, [z.data_ptr()])
    ccl.ccl_expert_dispatch(h, "bf16", rows, hidden, 2, [d_slots.ptr()], None, capacity, stream())
    ccl.ccl_comm_set_outputs(h, [dz.data_ptr()])
    ccl.ccl_expert_combine_grad(h, "bf16", rows, hidden, 2, [d_slots.ptr()], None, [z.data_ptr()], capacity, [dw.ptr()], stream())
    b = ccl.ccl_comm_create(1, [z.data_ptr()])
    ccl.ccl_comm_set_outputs(b, [back.ptr()])
    ccl.ccl_expert_combine(b, "bf16", rows, hidden, 2, [d_slots.ptr()], None, capacity, stream())
    for c in (h, b):
        ccl.ccl_comm_check(c)
        ccl.ccl_comm_destroy(c)
    for t in range(rows):
        of = [s for s in slots[0, t] if s >= 0]
        for s in of:
            assert torch.equal(z[s], tokens.t[t]) and torch.equal(dz[s], tokens.t[t])
        assert torch.equal(back.t[t], tokens.t[t] * len(of))
        size = float(tokens.t[t].double().square().sum())
        want = torch.tensor([size if s >= 0 else 0.0 for s in slots[0, t]], device="cuda", dtype=torch.float64)
        assert_within(dw.t[t], want, (hidden / 32 + 23) * U32 * want, "dweights")
    untouched = torch.ones(capacity, dtype=torch.bool, device="cuda")
    untouched[torch.from_numpy(slots[slots >= 0]).long()] = False
    assert not bool(z[untouched].any()) and back.guarded() and dw.guarded()


@pytest.mark.parametrize("rows", [4, 400])
def test_captured(rows):
    """Sort, dispatch, combine and its gradient in one graph, replayed on new choices; the same bits as calls one by one."""
    p, k, hidden, experts = 4, 3, 512, 10
    layer = Layer("bf16", p, rows, hidden, k, capacity=rows * k * p)
    ids = [torch.empty(rows, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    offsets = torch.empty(experts + p, dtype=torch.int32, device="cuda")
    there, back = layer.there, layer.back

    def step():
        ccl.ccl_expert_sort(there.h, rows, experts, k, [t.data_ptr() for t in ids], None, layer.capacity, ptrs(layer.slots),
                            offsets.data_ptr(), stream())
        layer.dispatch(there.h)
        layer.combine(back.h)
        layer.grad(there.h)

    def choose(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in ids:
            t.copy_(torch.randint(experts, t.shape, device="cuda", generator=g))

    outs = layer.to_expert + layer.to_tokens + layer.dweights
    choose(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        choose(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.t.clone() for a in outs]
        step()
        torch.cuda.synchronize()
        for a, x in zip(outs, got):
            assert torch.equal(a.t.view(torch.uint8), x.view(torch.uint8))
        want, _ = sort_by_expert(torch.stack(ids).cpu().numpy(), None, experts, layer.capacity)
        layer.slot = torch.from_numpy(want).cuda().long().view(p * rows, k)
        layer.check_tokens()
        layer.check_weights()
    for c in (there, back):
        with c:
            pass


@pytest.mark.parametrize("seed", range(20))
def test_random(seed):
    g = rng(500 + seed)
    p, k = int(g.choice([1, 2, 3, 8, 11])), int(g.integers(1, 10))
    hidden = int(np.exp(g.uniform(0, 8.5)))
    if g.random() < 0.6:
        hidden = -(-hidden // 8) * 8
    rows = int(np.exp(g.uniform(0, 5)))
    Layer(str(g.choice(["f32", "f16", "bf16"])), p, rows, hidden, k, capacity=int(rows * k * g.uniform(0.2, 2)) + 1,
          offset=int(g.choice([0, 0, 0, 1, 3])), weighted=bool(g.random() < 0.7), seed=seed).all()

"""ccl_expert_sort against the definition, choice by choice: every value is a
whole number and has to be equal."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import Array, Comm, ptrs, sort_by_expert, stream
from logit_testutil import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Choices:
    """A call's arrays on the device, and what it should write."""

    def __init__(self, ids, valid, experts, capacity, offset=0):
        p, rows, k = ids.shape
        self.ids, self.valid, self.experts, self.capacity = ids, valid, experts, capacity
        self.d_ids = [Array((rows, k), torch.int32, offset, torch.from_numpy(x)) for x in ids]
        self.d_valid = None if valid is None else [Array((rows,), torch.uint8, offset, torch.from_numpy(x)) for x in valid]
        self.slots = [Array((rows, k), torch.int32, offset) for _ in range(p)]
        self.offsets = Array((experts + p,), torch.int32, offset)
        self.buffers = [Array((4,), torch.float32) for _ in range(p)]
        self.comm = Comm(self.buffers)
        self.comm.arrays += self.slots + [self.offsets]

    def call(self, h):
        p, rows, k = self.ids.shape
        ccl.ccl_expert_sort(h, rows, self.experts, k, ptrs(self.d_ids), ptrs(self.d_valid), self.capacity, ptrs(self.slots),
                            self.offsets.ptr(), stream())

    def check(self):
        slots, offsets = sort_by_expert(self.ids, self.valid, self.experts, self.capacity)
        got = np.stack([s.t.cpu().numpy() for s in self.slots])
        assert np.array_equal(self.offsets.t.cpu().numpy(), offsets)
        assert np.array_equal(got, slots)


def run(ids, valid=None, experts=8, capacity=1 << 20, offset=0):
    c = Choices(ids, valid, experts, capacity, offset)
    with c.comm as h:
        c.call(h)
    c.check()


def random_ids(p, rows, k, experts, seed=0, bad=0.05):
    """Ids with favourites, some of them outside the experts."""
    g = rng(seed + 7 * p + rows + experts)
    ids = (g.random((p, rows, k)) ** 3 * experts).astype(np.int32)
    out = g.random((p, rows, k)) < bad
    return np.where(out, g.choice(np.array([-1, experts, 2 ** 31 - 1, -2 ** 31], dtype=np.int64), (p, rows, k)), ids).astype(np.int32)


@pytest.mark.parametrize("p, rows, k, experts", [
    (1, 1, 1, 1), (1, 1, 8, 64), (1, 31, 1, 3), (1, 33, 3, 5), (2, 5, 2, 1), (8, 3, 2, 5), (8, 16, 8, 256), (3, 100, 7, 61),
    (8, 200, 6, 64), (4, 1023, 3, 257), (1, 5000, 2, 1024), (1, 4097, 4, 1025), (2, 3001, 4, 4096), (64, 40, 4, 100),
    (9, 700, 5, 33), (8, 4096, 8, 256), (1, 70000, 2, 7), (64, 3, 2, 4096), (1, 2, 4096, 300)])
@pytest.mark.parametrize("padded", [False, True])
def test_sizes(p, rows, k, experts, padded):
    valid = (rng(rows).random((p, rows)) < 0.8).astype(np.uint8) * 255 if padded else None
    run(random_ids(p, rows, k, experts), valid, experts)


def sort_at_once(ids, valid, experts, capacity):
    """sort_by_expert's values by whole arrays, on the GPU: ids [p, rows, k], valid [p, rows] or None."""
    p, rows, k = ids.shape
    e = ids.reshape(-1).long()
    e = torch.where((e >= 0) & (e < experts), e, experts)
    if valid is not None:
        e = torch.where(valid.reshape(-1, 1).expand(-1, k).reshape(-1) != 0, e, experts)
    counts = torch.bincount(e, minlength=experts + 1)
    begin = counts.cumsum(0) - counts
    held = [experts // p + (r < experts % p) for r in range(p)]
    first = [sum(held[:r]) for r in range(p + 1)]
    owner = torch.tensor([r for r in range(p) for _ in range(held[r])] + [p - 1], device=e.device)
    base = torch.stack([begin[f] for f in first])
    order = torch.sort(e, stable=True).indices
    of = e[order]
    at = torch.arange(e.numel(), device=e.device) - base[owner[of]]
    slot = torch.where((of < experts) & (at < capacity), owner[of] * capacity + at, -1)
    slots = torch.empty_like(e).scatter_(0, order, slot).view(p, rows, k).int()
    offsets = [min(int(begin[x] - base[r]), capacity) for r in range(p) for x in range(first[r], first[r + 1] + 1)]
    return slots, torch.tensor(offsets, dtype=torch.int32, device=e.device)


@pytest.mark.parametrize("p, rows, k, experts", [(1, 2000003, 1, 16), (2, 700001, 3, 256), (1, 400001, 2, 4096), (8, 20011, 16, 1000), (3, 30000000, 2, 100)])
@pytest.mark.parametrize("padded", [False, True])
def test_long_lists(p, rows, k, experts, padded):
    """Stretches longer than a warp keeps in registers, up to 180 million choices."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    ids = (torch.rand(p, rows, k, device="cuda", generator=g) ** 2 * (experts + 1)).int() - (torch.rand(p, rows, k, device="cuda", generator=g) < 0.01).int()
    valid = (torch.rand(p, rows, device="cuda", generator=g) < 0.9).to(torch.uint8) if padded else None
    capacity = rows * k * 9 // 10
    slots = torch.full((p, rows, k), 7, dtype=torch.int32, device="cuda")
    offsets, buffers = Array((experts + p,), torch.int32), [Array((4,), torch.float32) for _ in range(p)]
    with Comm(buffers) as h:
        ccl.ccl_expert_sort(h, rows, experts, k, [t.data_ptr() for t in ids], None if valid is None else [t.data_ptr() for t in valid],
                            capacity, [t.data_ptr() for t in slots], offsets.ptr(), stream())
    want, want_offsets = sort_at_once(ids, valid, experts, capacity)
    assert torch.equal(offsets.t, want_offsets) and torch.equal(slots, want)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_alignment(offset):
    run(random_ids(3, 501, 5, 40), np.ones((3, 501), dtype=np.uint8), 40, offset=offset)


@pytest.mark.parametrize("p, rows, k, experts", [(1, 50, 2, 4), (4, 300, 4, 16), (8, 4000, 4, 64)])
@pytest.mark.parametrize("share", [0.0, 0.01, 0.5, 1.0])
def test_full_buffers(p, rows, k, experts, share):
    """Choices that find no row have slot -1, and the offsets end at the capacity."""
    run(random_ids(p, rows, k, experts), None, experts, capacity=int(share * rows * k))


@pytest.mark.parametrize("ids", ["one expert", "last expert", "none", "same choice twice", "descending"])
def test_lists(ids):
    p, rows, k, experts = 2, 2500, 4, 48
    full = {"one expert": np.zeros((p, rows, k)), "last expert": np.full((p, rows, k), experts - 1), "none": np.full((p, rows, k), -1),
            "same choice twice": np.repeat(random_ids(p, rows, 1, experts), k, 2),
            "descending": (-np.arange(p * rows * k) % experts).reshape(p, rows, k)}[ids].astype(np.int32)
    run(full, None, experts)


def test_no_valid_row():
    run(random_ids(2, 70, 3, 9), np.zeros((2, 70), dtype=np.uint8), 9)


@pytest.mark.parametrize("p, experts", [(1, 5), (3, 8), (64, 64)])
def test_no_rows(p, experts):
    """The offsets of nothing are 0."""
    offsets, buffers = Array((experts + p,), torch.int32), [Array((4,), torch.float32) for _ in range(p)]
    with Comm(buffers) as h:
        ccl.ccl_expert_sort(h, 0, experts, 2, None, None, 10, None, offsets.ptr(), stream())
    assert offsets.guarded() and not bool(offsets.t.any())


@pytest.mark.parametrize("rows", [3, 5000])
def test_graphs_that_share_a_communicator(rows):
    """Two graphs of one communicator's calls, replayed in turn with new ids, and a call between them."""
    a, b = (Choices(random_ids(4, rows, 4, 50, seed), None, 50, 1 << 20) for seed in (1, 2))
    with a.comm as h:
        a.call(h)
        torch.cuda.synchronize()
        graphs = []
        for c in (a, b):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                c.call(h)
        for seed in (3, 4):
            for c, g in zip((a, b), graphs):
                c.ids = random_ids(4, rows, 4, 50, seed + 10 * (c is b))
                for d, x in zip(c.d_ids, c.ids):
                    d.t.copy_(torch.from_numpy(x))
                g.replay()
            b.call(h)
        torch.cuda.synchronize()
        a.check()
        b.check()
    with b.comm:
        pass


def test_another_stream():
    c = Choices(random_ids(2, 900, 4, 30), None, 30, 1 << 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with c.comm as h, torch.cuda.stream(side):
        c.call(h)
    c.check()


@pytest.mark.parametrize("seed", range(24))
def test_random(seed):
    g = rng(1000 + seed)
    p = int(g.choice([1, 2, 3, 4, 8, 13]))
    rows, k, experts = int(np.exp(g.uniform(0, 8))), int(g.integers(1, 9)), int(np.exp(g.uniform(0, 7)))
    valid = (g.random((p, rows)) < 0.9).astype(np.uint8) if g.random() < 0.5 else None
    run(random_ids(p, rows, k, experts, seed, bad=0.1), valid, experts, capacity=int(rows * k * g.uniform(0.3, 3)))

"""The operators around layers from two streams at once: communicators are independent of one another, and one
communicator's calls may follow each other on different streams that are ordered by events."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from layer_testutil import ptrs, sort_by_expert
from test_expert_rows import Layer
from test_expert_sort import Choices, random_ids
from test_grads import Grads
from test_norm_e4m3 import Norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_two_communicators_at_once():
    """Everything that has scratch in its communicator, or waits, many times on two streams."""
    work = []
    for i in range(2):
        rows = (2500, 1001)[i]
        c = Choices(random_ids(4, rows, 3, 40, seed=i), np.ones((4, rows), dtype=np.uint8), 40, rows * 4)
        g = Grads([(300007, "bf16", 0), (70001, "f32", 0), (33, "f16", 1)] * 5, seed=i)
        n = Norm(("bf16", "f16")[i], 4, (3, 200)[i], 33000, 128)
        layer = Layer("bf16", 2, (300, 5)[i], 1001, 4, seed=i)
        work.append((c, g, n, layer))
    before = [[a.t.clone() for a in g.ins] for _, g, _, _ in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, (c, g, n, layer) in zip(streams, work):
            with torch.cuda.stream(s):
                c.call(c.comm.h)
                g.call(g.comm.h, 1.0)
                n.call(n.comm.h)
                layer.dispatch(layer.there.h)
                layer.grad(layer.there.h)
                layer.combine(layer.back.h)
    torch.cuda.synchronize()
    for (c, g, n, layer), old in zip(work, before):
        for comm in (c.comm, g.comm, n.comm, layer.there, layer.back):
            with comm:
                pass
        c.check()
        g.check(1.0, old)
        n.check()
        layer.check_rows()
        layer.check_tokens()
        layer.check_weights()


def test_one_communicator_over_ordered_streams():
    """Sort and gradient norm of one communicator, call by call on the other stream."""
    c = Choices(random_ids(2, 6000, 2, 64), None, 64, 15000)
    g = Grads([(500003, "f32", 0)] * 3)
    before = [a.t.clone() for a in g.ins]
    h = c.comm.h
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    last = None
    for i in range(40):
        s = streams[i % 2]
        if last is not None:
            s.wait_event(last)
        with torch.cuda.stream(s):
            if i % 4 < 2:
                c.call(h)
            else:
                g.call(h, 1.0)
            last = torch.cuda.Event()
            last.record(s)
    torch.cuda.synchronize()
    with c.comm, g.comm:
        pass
    c.check()
    g.check(1.0, before)


@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_norm_captured_on_a_side_stream(eps):
    """With eps 0 the call is two kernels."""
    n = Norm("f32", 2, 300, 1024, 0, eps=eps)
    n.call(n.comm.h)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        n.call(n.comm.h)
    for _ in range(2):
        n.x[0].t.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        n.check()
    for a in n.x:
        a.t[7] = 0.0
    n.res.t[7] = 1e-30
    n.res.t[7, 5] = 0.0
    n.before = n.res.t.clone()
    with n.comm:
        graph.replay()
        torch.cuda.synchronize()
        s = n.scales[0].t[:, 0]
        assert bool(torch.isnan(s[7])) == (eps == 0.0) and bool(torch.isfinite(s[:7]).all()) and bool(torch.isfinite(s[8:]).all())


def test_sort_then_rows_on_a_side_stream():
    """Slots written and used by kernels that may start early, behind another stream's work."""
    p, rows, k, experts, hidden = 2, 1500, 4, 10, 520
    layer = Layer("bf16", p, rows, hidden, k)
    ids = torch.randint(experts, (p, rows, k), dtype=torch.int32, device="cuda")
    offsets = torch.empty(experts + p, dtype=torch.int32, device="cuda")
    for a in layer.slots:
        a.t.fill_(-1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ccl.ccl_expert_sort(layer.there.h, rows, experts, k, [t.data_ptr() for t in ids], None, layer.capacity, ptrs(layer.slots),
                            offsets.data_ptr(), side.cuda_stream)
        layer.dispatch(layer.there.h)
        layer.combine(layer.back.h)
    torch.cuda.synchronize()
    want, ends = sort_by_expert(ids.cpu().numpy(), None, experts, layer.capacity)
    assert np.array_equal(offsets.cpu().numpy(), ends)
    layer.slot = torch.from_numpy(want).cuda().long().view(p * rows, k)
    with layer.there, layer.back:
        pass
    layer.check_rows()
    layer.check_tokens()

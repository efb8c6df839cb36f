"""The operators on experts' rows where their buffers lie differently between 16-byte boundaries, and the gradient of
dispatch.

Tolerances as in test_expert_rows: a weight's gradient is an fp32 sum over the columns, at most hidden / 32 + 8 products
in a thread and at most 15 more additions; its size is the sum of the products' sizes."""
import pytest
import torch

from layer_testutil import Array, Comm
from logit_testutil import rng
from test_expert_rows import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Mixed(Layer):
    """A layer whose tokens, experts' rows and the rows written of each lie `at` elements past a boundary, rank by rank."""

    def __init__(self, dtype, p, rows, hidden, k, at, weighted=True):
        super().__init__(dtype, p, rows, hidden, k, weighted=weighted)

        def moved(arrays, i):
            return [Array(tuple(a.t.shape), a.t.dtype, at[(i + r) % len(at)], a.t) for r, a in enumerate(arrays)]

        self.tokens, self.expert, self.to_tokens, self.to_expert = (
            moved(a, i) for i, a in enumerate((self.tokens, self.expert, self.to_tokens, self.to_expert)))
        self.there, self.back = Comm(self.tokens, self.to_expert), Comm(self.expert, self.to_tokens)
        self.there.arrays += self.slots + self.dweights + self.expert


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("at", [(0, 1), (1, 0, 2), (0, 3, 5), (0, 1, 2, 3, 4, 5, 6, 7), (4, 0), (0, 8, 1)])
@pytest.mark.parametrize("hidden", [8, 29, 64, 257, 1001, 4104])
def test_buffers_that_lie_differently(dtype, at, hidden):
    Mixed(dtype, 3, 13, hidden, 3, at).all()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("rows, hidden, k", [(4000, 61, 2), (2500, 303, 9), (1500, 1001, 1)])
def test_many_tokens(weighted, rows, hidden, k):
    Mixed("bf16", 2, rows, hidden, k, (0, 5, 2, 7), weighted).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p, rows, hidden, k", [(1, 1, 8, 1), (3, 40, 264, 3), (2, 30, 1001, 2), (8, 16, 2048, 8)])
def test_dispatch_gradient(dtype, p, rows, hidden, k):
    """row = w x: by the tokens combine of the rows' gradient; by the weights combine's gradient with the tokens where the
    tokens' gradient is and the rows' gradient where the experts' rows are.  Its rows are the forward's."""
    layer = Layer(dtype, p, rows, hidden, k)          # layer.expert: the gradient of the written rows
    with layer.there as h:
        layer.dispatch(h)
        torch.cuda.synchronize()
        forward = [a.t.clone() for a in layer.to_expert]
        for a, old in zip(layer.to_expert, layer.before):
            a.t.copy_(old)
        layer.grad(h)
    for a, x in zip(layer.to_expert, forward):
        assert torch.equal(a.t.view(torch.uint8), x.view(torch.uint8))
    layer.check_weights()                             # <x_t, gradient of the row>
    with layer.back as h:
        layer.combine(h)
    layer.check_tokens()                              # the sum of w times the gradient of the row


def test_dispatch_gradient_by_differences():
    """In whole numbers, where fp32 is exact: the slope of <rows, c> by each weight."""
    p, rows, hidden, k = 2, 4, 12, 2
    layer = Layer("f32", p, rows, hidden, k, capacity=9)
    g = rng(3)
    for arrays in (layer.tokens, layer.expert, layer.weights):
        for a in arrays:
            a.t.copy_(torch.from_numpy(g.integers(-4, 5, tuple(a.t.shape)).astype("float32")))
    with Comm(layer.tokens, layer.to_expert) as h:
        layer.grad(h)
    got = [a.t.clone() for a in layer.dweights]

    def value():
        for a in layer.to_expert:
            a.t.zero_()
        with Comm(layer.tokens, layer.to_expert) as h:
            layer.dispatch(h)
        return float(sum((a.t.double() * b.t.double()).sum() for a, b in zip(layer.to_expert, layer.expert)))

    for r in range(p):
        for i in range(rows * k):
            w = layer.weights[r].t.view(-1)
            old, ends = float(w[i]), []
            for step in (1.0, -1.0):
                w[i] = old + step
                ends.append(value())
            w[i] = old
            assert (ends[0] - ends[1]) / 2 == float(got[r].view(-1)[i])

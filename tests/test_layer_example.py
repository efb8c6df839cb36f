"""The example that runs the operators around layers together."""
import importlib.util
import os

import pytest
import torch

from logit_testutil import HALF_STEP, U32, assert_within

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer_step.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("expert_layer_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("p, rows, experts, k, group", [(1, 1, 3, 1, 64), (4, 6, 10, 3, 32), (8, 21, 5, 2, 128)])
def test_decode(example, p, rows, experts, k, group):
    """Each step's output against the layer in 64 bits on the same 8-bit input.  The experts' products are fp32 matrix products of
    256 terms (2 * 256 U32 of the terms' sizes, however they are summed), rounded to bf16, as is the weighted sum."""
    seen, w = example.decode(p=p, rows=rows, hidden=256, experts=experts, k=k, group=group)
    assert len(seen) == 3
    for s in seen:
        h = (sum(t.double() for t in s["partial"]).bfloat16().double() + s["residual"].double()).bfloat16()
        got = s["residual_out"]
        # the sum of p bf16 numbers in fp32 may round to another bf16 neighbour than that in fp64
        assert float((got.double() - h.double()).abs().max()) <= 2.0 ** -6 * float(h.double().abs().max())
        h = got.double()
        o = h * w["gamma"].double() / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
        top = o.view(rows, -1, group).abs().amax(2, keepdim=True).expand(-1, -1, group).reshape(rows, -1)
        assert bool(((s["x"].double() - o).abs() <= 2.0 ** -4 * o.abs() + top * (2.0 ** -10 / 448 + 1e-4)).all())
        x = s["x"].double()
        score = (s["x"] @ w["router"].t()).topk(k, 1)
        share = torch.softmax(score.values, 1).double()
        want, tol = torch.zeros(rows, 256, dtype=torch.float64, device="cuda"), torch.zeros(rows, 256, dtype=torch.float64, device="cuda")
        for j in range(k):
            a = w["weight"][score.indices[:, j]].double()
            want += share[:, j, None] * torch.bmm(x[:, None], a)[:, 0]
            size = share[:, j, None] * torch.bmm(x.abs()[:, None], a.abs())[:, 0]
            tol += size * (2 * 256 * U32 + HALF_STEP["bf16"] + (k + 8) * U32)
        assert_within(s["out"], want, tol + HALF_STEP["bf16"] * want.abs() * 1.01)


@pytest.mark.parametrize("p, rows, experts, k", [(1, 5, 4, 2), (4, 40, 7, 2), (3, 30, 8, 3), (8, 9, 5, 1)])
def test_training_gradients(example, p, rows, experts, k):
    """Loss, gradients, global norm and clipped gradients against autograd in 64 bits.  Gradients are sums of up to rows * p
    products of fp32 matrix products; 1e-5 of the largest gradient is some 100 U32 of it, and sums of 48 to 400 terms of
    mixed signs stay within that with room."""
    layer = example.Layer(p=p, rows=rows, experts=experts, k=k, max_norm=0.01)
    loss = layer.gradients()
    router = layer.router.double().requires_grad_()
    weight = torch.cat(layer.weight).double().requires_grad_()
    xs = [x.double().requires_grad_() for x in layer.x]
    n = sum(int(v.sum()) for v in layer.valid)
    total, mass, hits = 0.0, 0.0, torch.zeros(experts, device="cuda", dtype=torch.float64)
    for r in range(p):
        keep = layer.valid[r].bool()
        logits = xs[r] @ router.t()
        ids = layer.ids[r].long()
        share = torch.softmax(logits.gather(1, ids), 1)
        z = torch.tanh(torch.einsum("th,tkhg->tkg", xs[r], weight[ids]))
        y = xs[r] + (share[:, :, None] * z).sum(1)
        total = total + (y - layer.target[r].double())[keep].square().sum() / (n * layer.hidden)
        mass = mass + torch.softmax(logits, 1)[keep].sum(0)
        hits += torch.bincount(ids[keep].view(-1), minlength=experts)
    total = total + layer.coef * experts * (hits / (k * n) * mass / n).sum()
    total.backward()
    total = total.detach()
    assert abs(float(loss) - float(total)) <= 1e-5 * float(total)

    def near(got, want):
        assert float((got.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())

    for dr in layer.drouter:
        near(dr, router.grad)
    near(torch.cat(layer.dweight), weight.grad)
    for x, dx in zip(xs, layer.dx):
        near(dx, x.grad)
    before = [t.clone() for t in layer.drouter + layer.dweight]
    norm = float((router.grad.square().sum() + weight.grad.square().sum()).sqrt())
    layer.clip()
    got, factor = layer.norm.tolist()
    assert abs(got - norm) <= 1e-5 * norm
    assert abs(factor - min(1.0, 0.01 / (got + 1e-6))) <= 1e-6 * factor and factor < 1
    for t, old in zip(layer.drouter + layer.dweight, before):
        assert torch.equal(t, old * layer.norm[1])
    layer.step()
    layer.close()

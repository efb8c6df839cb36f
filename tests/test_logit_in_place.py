"""Communicators of which some ranks are in place and others are not, and
which of them the launchers are told are in place."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
import test_balance
import test_distill
import test_logit_rules
from ccl_testutil import ensure_built
from logit_testutil import Ranks, rng
from test_logit_refusals import A, CALLS, OK, front, status      # noqa: F401 (front: a fixture)


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


class Mixed(Ranks):
    """Every second rank is in place, from rank `first` on."""

    def __init__(self, parts, dtype, first=0, **layout):
        super().__init__(parts, dtype, **layout)
        self.same = [r for r in range(len(parts)) if r % 2 == first]
        for r in self.same:
            self.outs[r] = self.ins[r]
        ccl.ccl_comm_set_outputs(self.comm, [b.ptr() for b in self.outs])

    def finish(self, wrote=True):
        torch.cuda.synchronize()
        ccl.ccl_comm_check(self.comm)
        assert all(b.outside_untouched() for b in self.ins + self.outs)
        for r, (b, old) in enumerate(zip(self.ins, self.before)):
            if r not in self.same or not wrote:
                assert torch.equal(b.raw.view(torch.uint8), old.view(torch.uint8))
        ccl.ccl_comm_destroy(self.comm)


@pytest.mark.cpu
@pytest.mark.parametrize("op", CALLS)
def test_in_place_is_every_rank_in_place(front, op):             # noqa: F811
    for outputs, alias in (([1 * A, 2 * A], 1), ([3 * A, 4 * A], 0), ([1 * A, 4 * A], 0), ([3 * A, 2 * A], 0)):
        assert status(front, CALLS[op](front), outputs=outputs) == (OK, 1)
        assert front.fake_alias() == alias


@pytest.mark.cpu
def test_a_rank_without_columns_does_not_count(front):           # noqa: F811
    assert status(front, CALLS["rules"](front, vocab=1), outputs=[1 * A, 4 * A]) == (OK, 1)
    assert front.fake_alias()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,rows,vocab,layout", [(2, 5, 8190, {}), (4, 6, 8191, dict(offset=1)), (3, 40, 100003, dict(first=1)),
                                                 (4, 6, 3, {}), (16, 3, 2051, dict(offset=3, out_offset=1))])
def test_rules(gpu, monkeypatch, dtype, p, rows, vocab, layout):
    monkeypatch.setattr(test_logit_rules, "Ranks", Mixed)
    x = rng(p).normal(0, 4, (rows, vocab))
    test_logit_rules.check(x, p, dtype, test_logit_rules.make_rules(rows, vocab, 5, 200, 30, True), **layout)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", ["both", "each"])
@pytest.mark.parametrize("p,rows,vocab", [(2, 5, 8190), (4, 320, 3001), (16, 3, 2051)])
def test_distillation(gpu, monkeypatch, steps, p, rows, vocab):
    monkeypatch.setattr(test_distill, "Ranks", Mixed)
    g = rng(p)
    ids, t = test_distill.teacher(rows, vocab, 20, 4)
    test_distill.check(g.normal(0, 3, (rows, vocab)), ids, t, 1.5, p, "bf16", steps, weight=g.normal(0, 1, rows))


@pytest.mark.gpu
@pytest.mark.parametrize("E", [64, 61, 1500])
def test_balance_loss(gpu, monkeypatch, E):
    monkeypatch.setattr(test_balance, "Ranks", Mixed)
    xs = [rng(r).normal(0, 2, (300, E)) for r in range(3)]
    test_balance.check(xs, test_balance.choices(300, E, 3, 3, 6), "bf16", "both")

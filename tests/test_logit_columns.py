"""Rank buffers that are columns of one matrix: their rows lie between one
another's, and none overlaps another."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
import test_distill
import test_logit_rules
from ccl_testutil import ensure_built
from logit_testutil import GUARD, TORCH, rng
from test_logit_refusals import BAD, OK, ROWS, VOCAB, A, distill_call, front, rules_call, status      # noqa: F401 (front: a fixture)


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


CALLS = {"rules": rules_call, "distill": distill_call}
LEFT, RIGHT = 6, 5              # columns of the two ranks of the refusals' [4, 11] bf16 logits


@pytest.mark.cpu
@pytest.mark.parametrize("op", CALLS)
@pytest.mark.parametrize("ld,a,b,want", [
    (VOCAB, 0, LEFT, OK), (VOCAB + 5, 0, LEFT, OK), (VOCAB + 5, 0, LEFT + 3, OK),     # side by side
    (VOCAB, RIGHT, 0, OK), (VOCAB, RIGHT + VOCAB, 0, OK),                             # the other way round; a row further down
    (VOCAB, 0, LEFT + ROWS * VOCAB, OK), (VOCAB, 0, LEFT + (ROWS - 1) * VOCAB, OK),   # altogether below; the last row beside it
    (VOCAB, 0, LEFT - 1, BAD), (VOCAB, 1, LEFT, BAD), (VOCAB - 1, 0, LEFT, BAD),      # a column of both; a row that meets the next
    (VOCAB, 0, LEFT - 1 + (ROWS - 1) * VOCAB, BAD), (VOCAB, 0, LEFT + 1, BAD), (VOCAB + 1, RIGHT - 1, 0, BAD)])
def test_overlap_goes_by_rows(front, op, ld, a, b, want):        # noqa: F811
    """In place, and out of place over the columns of another matrix."""
    at = [8 * A + 2 * a, 8 * A + 2 * b]
    assert status(front, CALLS[op](front, ld=ld), inputs=at, outputs=at) == (want, int(want == OK))
    assert status(front, CALLS[op](front, ld=ld), outputs=at) == (want, int(want == OK))


@pytest.mark.cpu
def test_overlap_against_every_element(front):                   # noqa: F811
    g, seen = rng(1), [0, 0]
    for _ in range(2000):
        rows, ld = int(g.integers(1, 6)), int(g.integers(LEFT, 20))
        at = [8 * A + 2 * int(g.integers(0, 80)) for _ in range(2)]
        cells = [{x // 2 + i * ld + c for i in range(rows) for c in range(w)} for x, w in zip(at, (LEFT, RIGHT))]
        want = BAD if cells[0] & cells[1] else OK
        seen[want == OK] += 1
        assert status(front, rules_call(front, rows=rows, ld=ld, mask_rows=0, history_ld=0, history=0), outputs=at)[0] == want
    assert min(seen) > 200


@pytest.mark.cpu
@pytest.mark.parametrize("op", CALLS)
def test_an_output_between_an_inputs_rows(front, op):            # noqa: F811
    side = [8 * A, 8 * A + 2 * LEFT]
    assert status(front, CALLS[op](front, ld=VOCAB), inputs=side, outputs=side) == (OK, 1)
    assert status(front, CALLS[op](front, ld=VOCAB), inputs=side, outputs=side[::-1]) == (BAD, 0)     # another rank's input
    assert status(front, CALLS[op](front, ld=VOCAB), inputs=[8 * A, 9 * A], outputs=[8 * A + 2 * LEFT, 7 * A]) == (BAD, 0)   # six wide
    assert status(front, CALLS[op](front, ld=VOCAB + 1), inputs=[8 * A, 9 * A], outputs=[8 * A + 2 * LEFT, 7 * A]) == (OK, 1)


class Columns:
    """(as logit_testutil.Ranks, in place)  The parts beside one another in one [rows, ld] matrix."""

    def __init__(self, parts, dtype, ld=0, offset=0):
        p, rows = len(parts), parts[0].shape[0]
        raw = torch.full((GUARD + offset + rows * ld + GUARD,), float("nan"), dtype=TORCH[dtype], device="cuda")
        matrix = raw[GUARD + offset:].as_strided((rows, ld), (ld, 1))
        begin = np.cumsum([0] + [t.shape[1] for t in parts])[:-1]
        views = [matrix[:, b:b + t.shape[1]] for b, t in zip(begin, parts)]
        for v, t in zip(views, parts):
            v.copy_(t)
        self.views, self.raw, self.width = views, raw, int(sum(t.shape[1] for t in parts))
        self.rest = (raw, GUARD + offset, rows, ld)
        self.comm = ccl.ccl_comm_create(p, [v.data_ptr() for v in views])

    def output(self):
        return [v.double() for v in self.views]

    def finish(self, wrote=True):
        torch.cuda.synchronize()
        ccl.ccl_comm_check(self.comm)
        ccl.ccl_comm_destroy(self.comm)
        raw, start, rows, ld = self.rest
        seen = raw.clone()
        seen[start:].as_strided((rows, self.width), (ld, 1)).fill_(float("nan"))
        assert bool(torch.isnan(seen).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,rows,vocab,layout", [(3, 7, 8191, dict(ld=8191)), (4, 6, 8192, dict(ld=8192)), (2, 5, 999, dict(ld=1003, offset=1)),
                                                 (8, 40, 100003, dict(ld=100008)), (16, 3, 50, dict(ld=51))])
def test_rules(gpu, monkeypatch, dtype, p, rows, vocab, layout):
    monkeypatch.setattr(test_logit_rules, "Ranks", Columns)
    test_logit_rules.check(rng(p).normal(0, 4, (rows, vocab)), p, dtype, test_logit_rules.make_rules(rows, vocab, 5, 200, 30, True), **layout)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", ["forward", "both", "each"])
@pytest.mark.parametrize("p,rows,vocab,layout", [(3, 7, 8191, dict(ld=8191)), (4, 320, 3001, dict(ld=3003, offset=3)), (2, 30, 40000, dict(ld=40000)),
                                                 (16, 3, 2051, dict(ld=2051))])
def test_distillation(gpu, monkeypatch, steps, p, rows, vocab, layout):
    monkeypatch.setattr(test_distill, "Ranks", Columns)
    g = rng(p)
    ids, t = test_distill.teacher(rows, vocab, 20, 4)
    test_distill.check(g.normal(0, 3, (rows, vocab)), ids, t, 1.5, p, "bf16", steps, weight=g.normal(0, 1, rows), **layout)

"""Seeded random cases of the operators on logits: sizes, types, lists, and
rank buffers contiguous, strided, shifted, in place, in place in part, or the
columns of one matrix."""
import random

import pytest
import torch

import test_balance
import test_distill
import test_logit_rules
from ccl_testutil import ensure_built
from logit_testutil import Ranks, rng
from test_logit_columns import Columns
from test_logit_in_place import Mixed
from test_rules_biases import lists

pytestmark = pytest.mark.gpu

CASES = 25


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def log(r, lo, hi):
    return int(round(lo * (hi / lo) ** r.random()))


def layout(r, p, widest, vocab=0):
    """The class of the buffers, and where they lie; vocab: of a shard's columns, which may be strided."""
    stride = {"ld": widest + r.randint(0, 9)} if vocab and r.random() < 0.5 else {}
    kind = r.choice(["plain", "in place", "apart", "mixed", "columns"])
    if kind == "in place":
        return Ranks, dict(stride, in_place=True, offset=r.randint(0, 8))
    if kind == "apart":
        return Ranks, dict(stride, offset=[r.randint(0, 8) for _ in range(p)], out_offset=r.randint(0, 8))
    if kind == "mixed":
        return Mixed, dict(stride, offset=r.randint(0, 8), first=r.randint(0, 1))
    if kind == "columns" and vocab >= p:
        return Columns, dict(ld=vocab + r.randint(0, 9), offset=r.randint(0, 8))
    return Ranks, stride


def shape(r):
    p = r.choice([1, 2, 3, 4, 5, 8, 8, 11, 16, 33, 64])
    vocab = log(r, 1, 200000)
    return p, vocab, log(r, 1, max(2, min(500, 3000000 // vocab)))


@pytest.mark.parametrize("seed", range(6))
def test_rules(monkeypatch, seed):
    for i in range(CASES):
        r, g = random.Random(1000 * seed + i), rng(1000 * seed + i)
        p, vocab, rows = shape(r)
        cls, where = layout(r, p, -(-vocab // p), vocab)
        monkeypatch.setattr(test_logit_rules, "Ranks", cls)
        rules = test_logit_rules.make_rules(rows, vocab, i, r.choice([0, log(r, 1, 20000)]), r.choice([0, log(r, 1, 600)]), r.random() < 0.6)
        if r.random() < 0.2:
            rules = test_logit_rules.Rules(**dict(rules.h, **lists(g, rows, vocab, log(r, 300, 5000))))
        test_logit_rules.check(g.normal(0, 4, (rows, vocab)), p, r.choice(["bf16", "f16", "f32"]), rules, **where)


@pytest.mark.parametrize("seed", range(6))
def test_distillation(monkeypatch, seed):
    for i in range(CASES):
        r, g = random.Random(2000 * seed + i), rng(2000 * seed + i)
        p, vocab, rows = shape(r)
        cls, where = layout(r, p, -(-vocab // p), vocab)
        monkeypatch.setattr(test_distill, "Ranks", cls)
        k = min(log(r, 1, 1024), vocab)
        ids, t = test_distill.teacher(rows, vocab, k, i)
        test_distill.check(g.normal(0, 3, (rows, vocab)), ids, t, r.choice([0.3, 1.0, 2.0, 5.0]), p, r.choice(["bf16", "f16", "f32"]),
                           r.choice(["both", "forward", "each"]), weight=g.normal(0, 1, rows) if r.random() < 0.6 else None,
                           teacher_dtype=r.choice(["f32", "bf16", "f16"]), **where)


@pytest.mark.parametrize("seed", range(6))
def test_balance_loss(monkeypatch, seed):
    for i in range(CASES):
        r, g = random.Random(3000 * seed + i), rng(3000 * seed + i)
        p, E = shape(r)[0], log(r, 1, 1300)
        rows = log(r, 1, max(2, min(6000, 3000000 // (E * p))))
        cls, where = layout(r, p, E)
        monkeypatch.setattr(test_balance, "Ranks", cls)
        far = r.choice([0, 0, 50, -3000, 1e5])
        test_balance.check([g.normal(0, 2, (rows, E)) + far for _ in range(p)], test_balance.choices(rows, E, r.randint(1, min(E, 9)), p, i),
                           r.choice(["bf16", "f16", "f32"]), r.choice(["both", "forward", "each"]),
                           test_balance.padding(rows, p, i) if r.random() < 0.5 else None, **where)

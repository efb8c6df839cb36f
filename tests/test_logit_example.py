"""The example that runs the operators on logits together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sharded_head_step.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("sharded_head_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("p, rows, vocab", [(1, 1, 500), (4, 3, 1003)])
def test_decode_stays_in_the_grammar_and_repeats_itself(example, p, rows, vocab):
    tokens, allowed = example.decode(p=p, rows=rows, vocab=vocab)
    assert tokens.shape == (rows, 8)
    assert allowed.gather(1, tokens.long()).all()
    again, _ = example.decode(p=p, rows=rows, vocab=vocab)
    assert torch.equal(tokens, again)


def test_training_lowers_both_losses(example):
    seen = example.train()
    assert all(d >= 0 and b > 0 for d, b in seen)
    assert seen[-1][0] < seen[0][0]
    assert seen[-1][1] < seen[0][1]

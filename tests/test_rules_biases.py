"""GPU tests of long bias lists through ccl_logit_rules: more entries in a
slice of the columns than a CTA keeps."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import Ranks, rng, shards, stream
from test_logit_rules import Rules, check, make_rules

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def lists(g, rows, vocab, most, hot=0.3):
    """Rows of no, few and up to `most` entries; some tokens come again and again, some are outside the vocabulary."""
    n = np.array([(0, 3, most // 2, most)[i % 4] for i in range(rows)])
    total = int(n.sum())
    tokens = g.integers(-2, vocab + 2, total)
    tokens = np.where(g.random(total) < hot, g.integers(0, min(vocab, 40), total) * max(1, vocab // 40), tokens)
    return {"bias_offsets": np.concatenate([[0], np.cumsum(n)]).astype(np.int32), "bias_tokens": tokens.astype(np.int32),
            "bias_values": g.normal(0, 2, total).astype(np.float32)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,rows,vocab,most,layout", [
    (1, 4, 9000, 9000, {}), (2, 4, 5003, 20000, dict(offset=3)), (1, 40, 150001, 6000, {}), (3, 8, 100003, 30000, dict(in_place=True)),
    (2, 40, 150001, 4000, dict(in_place=True, offset=1)), (1, 4, 100, 3000, {})])
def test_long_lists_beside_histories_and_masks(dtype, p, rows, vocab, most, layout):
    a = make_rules(rows, vocab, 7, 500, 0, True).h
    g = rng(most)
    a.update(lists(g, rows, vocab, most))
    check(g.normal(0, 4, (rows, vocab)), p, dtype, Rules(**a), **layout)


@pytest.mark.parametrize("dense", [False, True])
def test_entries_of_one_token_add_in_list_order(dense):
    """Sums that another order would round differently, bit for bit; the logits themselves are 0."""
    g = rng(3)
    vocab, n = 5000, 12000
    tokens = (g.integers(0, vocab, n) if dense else g.integers(0, 30, n) * 150).astype(np.int32)
    values = (g.normal(0, 1, n) * 10.0 ** g.integers(-3, 4, n)).astype(np.float32)
    want = np.zeros(vocab, dtype=np.float32)
    for t, v in zip(tokens, values):
        want[t] = np.float32(want[t] + v)
    rules = Rules(bias_offsets=np.array([0, n], dtype=np.int32), bias_tokens=tokens, bias_values=values)
    ranks = Ranks(shards(torch.zeros(1, vocab, device="cuda"), 1), "f32")
    ccl.ccl_logit_rules(ranks.comm, "f32", 1, vocab, rules.s, stream=stream())
    torch.cuda.synchronize()
    assert np.array_equal(ranks.outs[0].view.cpu().numpy()[0], want)
    ranks.finish()


def test_time_goes_with_the_length_of_the_list():
    """Ten times the entries, for ten times the tokens, may not take the hundredfold time."""
    rows, vocab = 64, 32000
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    comm = ccl.ccl_comm_create(1, [x.data_ptr()])
    ccl.ccl_comm_set_outputs(comm, [y.data_ptr()])

    def us(n):
        tokens = np.stack([rng(i).permutation(vocab)[:n] for i in range(rows)]).astype(np.int32).reshape(-1)
        rules = Rules(bias_offsets=(np.arange(rows + 1) * n).astype(np.int32), bias_tokens=tokens,
                      bias_values=np.ones(rows * n, dtype=np.float32))
        times = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ccl.ccl_logit_rules(comm, "bf16", rows, vocab, rules.s, stream=stream())
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        assert bool((y.float().sum(1) == n).all())
        return min(times)

    few, many = us(vocab // 10), us(vocab)
    ccl.ccl_comm_destroy(comm)
    print(f"{few:.0f} us, {many:.0f} us")
    assert many < 30 * few, (few, many)

"""GPU tests of roundings that the operators on logits do not make."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import Ranks, rng, shards, stream
from test_logit_rules import Rules

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_repetition_divides_once(in_place, biased):
    """The rules in fp32 as the header writes them, one rounding a step, bit for bit: sum of biases, quotient or product,
    two differences (frequency * c is a rounding of its own)."""
    rows, vocab, n = 40, 3000, 2500
    g = rng(1)
    f = np.float32
    x = g.normal(0, 4, (rows, vocab)).astype(f)
    history = g.integers(0, vocab, (rows, n)).astype(np.int32)
    prompt = g.integers(0, n, rows).astype(np.int32)
    rep, freq, pres = (g.uniform(a, b, rows).astype(f) for a, b in ((0.6, 2.0), (-1, 1), (-1, 1)))
    arrays = dict(history=history, prompt_len=prompt, repetition=rep, frequency=freq, presence=pres)
    want = x.copy()
    if biased:
        arrays.update(bias_offsets=(np.arange(rows + 1) * 2000).astype(np.int32), bias_values=g.normal(0, 3, rows * 2000).astype(f),
                      bias_tokens=np.concatenate([g.permutation(vocab)[:2000] for _ in range(rows)]).astype(np.int32))
        for i in range(rows):
            at = slice(2000 * i, 2000 * (i + 1))
            want[i, arrays["bias_tokens"][at]] += arrays["bias_values"][at]       # no token twice
    for i in range(rows):
        seen = np.unique(history[i])
        want[i, seen] = np.where(want[i, seen] > 0, want[i, seen] / rep[i], want[i, seen] * rep[i])
        made, times = np.unique(history[i, prompt[i]:], return_counts=True)
        want[i, made] = (want[i, made] - freq[i] * times.astype(f)) - pres[i]
    assert want.dtype == f
    ranks = Ranks(shards(torch.from_numpy(x).cuda(), 2), "f32", in_place=in_place)
    ccl.ccl_logit_rules(ranks.comm, "f32", rows, vocab, Rules(**arrays).s, stream=stream())
    torch.cuda.synchronize()
    got = torch.cat([b.view for b in ranks.outs], 1).cpu().numpy()
    ranks.finish()
    differ = got.view(np.int32) != want.view(np.int32)
    assert not differ.any(), f"{int(differ.sum())} of {differ.size} values"

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


def one_hot_case(rows, E, k, p, seed, even):
    """Router rows of one finite logit each: their softmax is exactly 1 there, so the loss is sum_t a_e(t), and what is
    left to round are the coefficients, the sums and the result."""
    g = rng(seed)
    at = [g.integers(0, E // 2, rows) for _ in range(p)]           # (a dropped or doubled row of these changes the loss)
    xs = []
    for a in at:
        x = np.full((rows, E), -np.inf, dtype=np.float32)
        x[np.arange(rows), a] = g.normal(0, 5, rows)
        xs.append(x)
    if even:        # nearly equal counts: next to the mean the differences are small
        ids = [(np.arange(rows * k) % E).reshape(rows, k).astype(np.int32) for _ in range(p)]
    else:           # the first half of the experts has two thirds of the choices
        ids = [np.where(g.random((rows, k)) < 2 / 3, g.integers(0, E // 2, (rows, k)), g.integers(E // 2, E, (rows, k))).astype(np.int32)
               for _ in range(p)]
    return xs, at, ids


@pytest.mark.parametrize("p,rows,E,k", [(1, 7, 64, 2), (2, 1000, 64, 4), (3, 4001, 61, 3), (8, 2100, 96, 1), (4, 10000, 128, 2), (2, 50, 1500, 8),
                                        (8, 5000, 33, 4), (1, 30000, 8, 1)])
@pytest.mark.parametrize("even", [False, True])
def test_the_loss_misses_no_row_and_is_rounded_once(p, rows, E, k, even):
    """loss = n mean(a) + sum_t d_e(t).  The first term is fp64.  d_e = fl(E count - sum) fl(scale): three roundings; over the row's
    one exponential and its reciprocal (two ulps, 4 u): six more.  A thread adds the d of its own rows in fp32, at most m of them,
    then five steps of a warp; the rest is fp64.  So the sum of d is off by at most (14 + m) u sum |d|, a small part of one row's |d|,
    which the test sees to; the loss is rounded once more."""
    worst = 0.0
    for seed in range(6):
        xs, at, ids = one_hot_case(rows, E, k, p, seed, even)
        coef = float(np.float32(0.01 * (1 + seed / 7)))
        n = p * rows
        counts = sum(np.bincount(i.reshape(-1), minlength=E) for i in ids)
        scale = coef * E / (k * float(n) ** 2)
        d = (counts - counts.mean()) * scale
        picked = [d[a] for a in at]
        want = n * (counts.mean() * scale) + sum(float(v.sum()) for v in picked)
        # a CTA has eight warps, and there are at least two CTAs an SM and 8 rows a CTA: a thread has at most this many rows
        m = -(-rows * p // (152 * 8)) + 1
        size = sum(float(np.abs(v).sum()) for v in picked)
        off = (14 + m) * 2.0 ** -24 * size
        if not even:
            assert off < 0.25 * min(float(np.abs(v).min()) for v in picked), "the tolerance has to tell a row"
        ranks = Ranks([torch.from_numpy(x).cuda() for x in xs], "f32")
        ids_d = [torch.from_numpy(i).cuda() for i in ids]
        cnt, tok = torch.empty(p, E, dtype=torch.int32, device="cuda"), torch.empty(p, dtype=torch.int32, device="cuda")
        loss = torch.empty(1, device="cuda")
        ccl.ccl_balance_loss(ranks.comm, "f32", "forward", rows, E, k, [i.data_ptr() for i in ids_d], None, coef, 0, cnt.data_ptr(),
                             tok.data_ptr(), loss.data_ptr(), stream=stream())
        torch.cuda.synchronize()
        err = abs(float(loss) - want)
        # half a step of the result, and 2^-40 for the fp64 sums
        assert err <= (2.0 ** -24 + 2.0 ** -40) * abs(want) + off, (seed, err / abs(want) * 2 ** 24, off / abs(want) * 2 ** 24)
        worst = max(worst, (err - off) / abs(want) * 2 ** 24)
        ranks.finish(wrote=False)
    print(f"worst beyond the sums: {worst:.2f} u")


@pytest.mark.parametrize("E", list(range(2, 65)) + [100, 203, 511, 600, 700, 999, 1001, 1024])
def test_the_softmax_divides_once(E):
    """Rows of equal logits, coefficients that fp32 holds exactly and that add up to 0: each probability is fl(1 / E), each
    gradient one product with it, bit for bit."""
    rows, n = 64, 64
    g = rng(E)
    ids = np.minimum(g.integers(0, E, (rows, 1)), g.integers(0, E, (rows, 1))).astype(np.int32)
    d = (E * np.bincount(ids.reshape(-1), minlength=E) - n) / float(n) ** 2          # coef E count / (k n^2) - its mean, k = coef = 1
    assert np.abs(d).sum() * n ** 2 < 2 ** 24
    want = d.astype(np.float32) * (np.float32(1) / np.float32(E))
    for layout in (dict(), dict(offset=1)):
        ranks = Ranks([torch.zeros(rows, E, device="cuda")], "f32", **layout)
        ids_d = torch.from_numpy(ids).cuda()
        cnt, tok = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        loss = torch.empty(1, device="cuda")
        ccl.ccl_balance_loss(ranks.comm, "f32", "both", rows, E, 1, [ids_d.data_ptr()], None, 1.0, 0, cnt.data_ptr(), tok.data_ptr(),
                             loss.data_ptr(), stream=stream())
        torch.cuda.synchronize()
        got = ranks.outs[0].view.cpu().numpy()
        ranks.finish()
        assert np.array_equal(got.view(np.int32), np.broadcast_to(want, got.shape).view(np.int32))


@pytest.mark.parametrize("steps", ["both", "each"])
def test_the_teachers_softmax_divides_once(steps):
    """Equal teacher logits, at tokens whose own probability is 0 in fp32: each gradient is -fl(1 / k), bit for bit, for every
    number of entries at once (row i has i + 1)."""
    rows = k = 300
    z = torch.zeros(rows, 1000, device="cuda")
    z[:, 500:] = -200.0
    ids = torch.where(torch.arange(k, device="cuda") <= torch.arange(rows, device="cuda")[:, None],
                      600 + torch.arange(k, device="cuda"), -1).to(torch.int32)
    t, loss, stats = torch.full((rows, k), 3.0, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    ranks = Ranks(shards(z, 2), "f32")
    for s in {"both": ["both"], "each": ["forward", "backward"]}[steps]:
        ccl.ccl_distill_topk(ranks.comm, "f32", s, rows, 1000, k, ids.data_ptr(), t.data_ptr(), loss=loss.data_ptr(),
                             stats=stats.data_ptr(), stream=stream())
    torch.cuda.synchronize()
    got = torch.cat([b.view for b in ranks.outs], 1)[:, 600:600 + k].cpu().numpy()
    ranks.finish()
    want = np.where(ids.cpu().numpy() >= 0, -(np.float32(1) / np.arange(1, rows + 1, dtype=np.float32))[:, None], np.float32(0))
    assert np.array_equal(got, want), f"{int((got != want).any(1).sum())} rows"


def test_differences_of_the_counts_are_rounded_once():
    """Two experts, equal logits, counts given: the gradient is half of d_e = coef (2 count_e - n) / n^2, the other's with the
    other sign, so what is seen is d_e itself: the fp64 value rounded to fp32."""
    g = rng(5)
    x = torch.zeros(1, 2, device="cuda")
    y = torch.empty_like(x)
    comm = ccl.ccl_comm_create(1, [x.data_ptr()])
    ccl.ccl_comm_set_outputs(comm, [y.data_ptr()])
    got, want = [], []
    for _ in range(300):
        n = int(2 ** g.uniform(1, 30.9))
        c0 = int(g.integers(0, n + 1))
        coef = float(np.float32(10 ** g.uniform(-4, 1)))
        counts = torch.tensor([c0, n - c0], dtype=torch.int32, device="cuda")
        tokens = torch.tensor([n], dtype=torch.int32, device="cuda")
        ccl.ccl_balance_loss(comm, "f32", "backward", 1, 2, 1, None, None, coef, 0, counts.data_ptr(), tokens.data_ptr(), 0, stream=stream())
        got.append(2 * y[0].cpu().numpy())
        d = (2 * c0 - n) * (coef / float(n) ** 2)
        want.append(np.array([d, -d]).astype(np.float32))
    ccl.ccl_comm_destroy(comm)
    got, want = np.stack(got), np.stack(want)
    # (fp64's own roundings may turn a tie: one in 2^27)
    off = got != want
    assert off.sum() == 0, f"{int(off.any(1).sum())} of 300, by up to {float(np.abs(got / want - 1)[off].max() * 2 ** 24):.2f} u"

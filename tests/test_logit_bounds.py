"""The checked build's tests of the accesses that the operators on logits make
(include/ccl.h, ccl_bounds_checked).  The debug hook has the checks take every
rank buffer, and every list with an entry a row, for one row shorter than the
call says: the last row's accesses are then recorded and not made, and the
other rows come out as ever.  These tests run only against the checked library
(test_zy_checked_logit_bounds.py runs them against it)."""
import os

import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from logit_testutil import Ranks, rng, shards, stream
from test_logit_rules import make_rules

if "CCL_LIBRARY" not in os.environ:
    pytest.skip("the default build has no bounds checks (CCL_LIBRARY selects the checked build)", allow_module_level=True)

pytestmark = pytest.mark.gpu

LAYOUTS = [dict(), dict(offset=1), dict(offset=3, out_offset=1), dict(in_place=True), dict(in_place=True, offset=5)]


@pytest.fixture(scope="module", autouse=True)
def _checked():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ccl.load_library()
    if not ccl.ccl_bounds_checked():
        pytest.skip("the default build has no bounds checks (CCL_LIBRARY selects the checked build)")


def bits(t):
    return t.contiguous().view(torch.uint8)


def violated(ranks, call, site):
    """Runs `call` with the hook; the record, and that the outputs' last rows are what they were.  Their other rows."""
    before = [b.view.clone() for b in ranks.outs]
    ccl.ccl_comm_set_debug(ranks.comm, 0, 2)
    call()
    with pytest.raises(ccl.CclError) as e:
        ccl.ccl_comm_check(ranks.comm)
    assert e.value.status == ccl.CCL_ERR_BOUNDS and f"site {site}" in str(e.value)
    ccl.ccl_comm_set_debug(ranks.comm, 0, 0)
    for b, old in zip(ranks.outs, before):
        assert torch.equal(bits(b.view[-1]), bits(old[-1]))
    return [b.view[:-1].clone() for b in ranks.outs]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,vocab", [(6, 8190), (40, 150001), (3, 5)])
def test_rules(dtype, layout, rows, vocab):
    full = torch.from_numpy(rng(rows).normal(0, 4, (rows, vocab))).cuda()
    rules = make_rules(rows, vocab, 5, 300, 40, True)
    call = lambda r: ccl.ccl_logit_rules(r.comm, dtype, rows, vocab, rules.s, stream=stream())
    ranks = Ranks(shards(full, 2), dtype, **layout)
    got = violated(ranks, lambda: call(ranks), 8)
    ranks.finish()
    ranks = Ranks(shards(full, 2), dtype, **layout)
    call(ranks)
    torch.cuda.synchronize()
    for b, g in zip(ranks.outs, got):
        assert torch.equal(bits(b.view[:-1]), bits(g))
    ranks.finish()


@pytest.mark.parametrize("what", ["history", "mask", "repetition"])
def test_one_rule_alone(what):
    """Lists are tested too, and not by the logits' own checks alone."""
    rows, vocab = 4, 3000
    h = make_rules(rows, vocab, 5, 300, 40, True).h
    arrays = {"history": ("history", "history_len", "frequency"), "mask": ("mask", "mask_index"), "repetition": ("history", "repetition")}[what]
    from test_logit_rules import Rules
    rules = Rules(**{k: h[k] for k in arrays})
    ranks = Ranks(shards(torch.zeros(rows, vocab, device="cuda"), 1), "f32")
    violated(ranks, lambda: ccl.ccl_logit_rules(ranks.comm, "f32", rows, vocab, rules.s, stream=stream()), 8)
    ranks.finish()


@pytest.mark.parametrize("steps", ["forward", "backward", "both"])
@pytest.mark.parametrize("layout", LAYOUTS + [dict(ld=60000)])
@pytest.mark.parametrize("p,rows,vocab,k", [(2, 5, 8190, 20), (2, 170, 100003, 200), (8, 330, 8003, 40), (1, 3, 7, 2)])
def test_distillation(steps, layout, p, rows, vocab, k):
    g = rng(vocab)
    full = torch.from_numpy(g.normal(0, 3, (rows, vocab))).cuda()
    ids = torch.from_numpy(g.integers(-1, vocab, (rows, k)).astype(np.int32)).cuda()
    t, w = torch.from_numpy(g.normal(0, 3, (rows, k))).cuda().float(), torch.ones(rows, device="cuda")

    def run(loss, stats, broken):
        ranks = Ranks(shards(full, p), "bf16", **layout)
        call = lambda: ccl.ccl_distill_topk(ranks.comm, "bf16", steps, rows, vocab, k, ids.data_ptr(), t.data_ptr(), temperature=2.0,
                                            row_weight=w.data_ptr(), loss=loss.data_ptr(), stats=stats.data_ptr(), ld=layout.get("ld", 0),
                                            stream=stream())
        if broken:
            out = violated(ranks, call, 9)
        else:
            call()
            torch.cuda.synchronize()
            out = [b.view[:-1].clone() for b in ranks.outs]
        ranks.finish(wrote=steps != "forward")
        return out

    stats = [torch.full((rows, 2), 1.5, device="cuda") for _ in range(2)]
    loss = [torch.full((rows,), 1.5, device="cuda") for _ in range(2)]
    got, want = run(loss[0], stats[0], True), run(loss[1], stats[1], False)
    for a, b in zip(got + [loss[0][:-1], stats[0][:-1]], want + [loss[1][:-1], stats[1][:-1]]):
        assert torch.equal(bits(a), bits(b))
    assert float(loss[0][-1]) == 1.5 and bool((stats[0][-1] == 1.5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("steps", ["forward", "backward", "both"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("p,rows,E,k", [(2, 20, 64, 4), (8, 3000, 64, 6), (2, 50, 61, 3), (3, 4000, 33, 2), (1, 40, 700, 2), (2, 30, 1500, 4)])
@pytest.mark.parametrize("padded", [False, True])
def test_balance_loss(dtype, steps, layout, p, rows, E, k, padded):
    """(All rows' gradients hang on the last row's choices: that it is recorded and left alone is what is tested.)"""
    g = rng(E)
    ranks = Ranks([torch.from_numpy(g.normal(0, 2, (rows, E))).cuda() for _ in range(p)], dtype, **layout)
    ids = [torch.from_numpy(g.integers(0, E, (rows, k)).astype(np.int32)).cuda() for _ in range(p)]
    valid = [torch.ones(rows, dtype=torch.uint8, device="cuda") for _ in range(p)]
    counts, tokens = torch.ones(p, E, dtype=torch.int32, device="cuda"), torch.full((p,), rows, dtype=torch.int32, device="cuda")
    loss = torch.empty(1, device="cuda")
    call = lambda: ccl.ccl_balance_loss(ranks.comm, dtype, steps, rows, E, k, [t.data_ptr() for t in ids],
                                        [t.data_ptr() for t in valid] if padded else None, 0.01, 0, counts.data_ptr(), tokens.data_ptr(),
                                        loss.data_ptr(), stream=stream())
    violated(ranks, call, 10)
    if steps != "backward":
        assert int(counts.sum()) == p * (rows - 1) * k and tokens.tolist() == [rows - 1 if padded else rows] * p
    call()
    ccl.ccl_comm_check(ranks.comm)
    if steps != "backward":
        assert int(counts.sum()) == p * rows * k and tokens.tolist() == [rows] * p
    ranks.finish(wrote=steps != "forward")

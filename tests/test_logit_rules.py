"""GPU tests of ccl_logit_rules against a plain fp64 evaluation, row by row."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import (FLOOR, HALF_STEP, TORCH, U32, Ranks, assert_within, ptr, rng, shards, stream)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


class Rules:
    """Host copies of a call's rules, and the structure with their device arrays."""

    def __init__(self, **arrays):
        self.mask = arrays.get("mask")
        self.h = arrays
        self.d = {}
        for k, v in arrays.items():
            if v is not None:
                self.d[k] = torch.from_numpy(np.ascontiguousarray(v)).cuda()
        s = ccl.LogitRules(**{k: v.data_ptr() for k, v in self.d.items()})
        if "history" in self.d:
            s.history_ld = self.h["history"].shape[1]
        if "bias_tokens" in self.d:
            s.bias_count = len(self.h["bias_tokens"])
        if "mask" in self.d:
            s.mask_rows, s.mask_ld = self.h["mask"].shape
        self.s = s


def make_rules(rows, vocab, seed, history=0, bias=0, mask=False, penalties=True):
    g = rng(seed)
    a = {}
    if history:
        a["history"] = (g.random((rows, history)) ** 3 * vocab).astype(np.int32)
        a["history"][g.random((rows, history)) < 0.02] = -1              # no token
        a["history"][g.random((rows, history)) < 0.02] = vocab           # past the vocabulary
        a["history_len"] = g.integers(-1, history + 3, rows).astype(np.int32)
        a["history_len"][-1] = history
        a["prompt_len"] = g.integers(-1, history + 3, rows).astype(np.int32)
    if penalties:
        a["repetition"] = (0.7 + g.random(rows)).astype(np.float32)
        a["frequency"] = (g.random(rows) - 0.3).astype(np.float32)
        a["presence"] = (g.random(rows) - 0.3).astype(np.float32)
    if bias:
        n = g.integers(0, bias + 1, rows)
        a["bias_offsets"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        total = max(1, int(n.sum()))
        a["bias_tokens"] = g.integers(-1, min(vocab, 3 * bias) + 1, total).astype(np.int32)   # many twice, some outside
        a["bias_values"] = g.normal(0, 3, total).astype(np.float32)
    if mask:
        words = (vocab + 31) // 32 + 1
        keep = np.array([0.0, 0.02, 0.98, 1.0])[np.arange(rows) % 4]
        bits = g.random((rows, words * 32)) < keep[:, None]
        a["mask"] = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
        a["mask_index"] = g.integers(-1, rows + 1, rows).astype(np.int32)    # -1 and rows: no mask
    return Rules(**a)


def exact(x, rules):
    """(y, bound on the fp32 evaluation's error before the last rounding), fp64."""
    h = rules.h
    y, off = x.copy(), np.zeros_like(x)
    rows, vocab = x.shape
    for i in range(rows):
        top = np.abs(np.where(np.isfinite(x[i]), x[i], 0.0))   # the largest magnitude an element passes through
        steps = np.zeros(vocab)                                # fp32 roundings it meets
        if "bias_tokens" in h:
            n = len(h["bias_tokens"])
            for k in range(*np.clip(h["bias_offsets"][i:i + 2], 0, n)):
                v = h["bias_tokens"][k]
                if 0 <= v < vocab:
                    y[i, v] += float(h["bias_values"][k])
                    top[v] += abs(float(h["bias_values"][k]))
                    steps[v] += 1
        if "history" in h:
            tokens = h["history"][i]
            n = len(tokens) if "history_len" not in h else int(np.clip(h["history_len"][i], 0, len(tokens)))
            start = 0 if "prompt_len" not in h else max(0, int(h["prompt_len"][i]))
            ok = lambda t: t[(t >= 0) & (t < vocab)]
            every, made = np.unique(ok(tokens[:n])), ok(tokens[start:n])
            if "repetition" in h:
                r = float(h["repetition"][i])
                y[i, every] = np.where(y[i, every] > 0, y[i, every] / r, y[i, every] * r)
                top[every] *= max(r, 1 / r)
                steps[every] += 1
            made, times = np.unique(made, return_counts=True)
            for name, by in (("frequency", times), ("presence", np.ones_like(times))):
                if name in h:
                    d = float(h[name][i]) * by
                    y[i, made] -= d
                    top[made] += np.abs(d)
                    steps[made] += 2
        off[i] = steps * U32 * top
        if "mask" in h:
            m = h["mask_index"][i] if "mask_index" in h else i
            if 0 <= m < len(h["mask"]):
                bits = np.unpackbits(h["mask"][m].view(np.uint8), bitorder="little")[:vocab]
                y[i, bits == 0] = -np.inf
    return y, off


def run(x, p, dtype, rules, **layout):
    full = torch.from_numpy(x).cuda().to(TORCH[dtype])
    ranks = Ranks(shards(full, p), dtype, **layout)
    rows, vocab = x.shape
    ccl.ccl_logit_rules(ranks.comm, dtype, rows, vocab, rules.s, ld=layout.get("ld", 0), stream=stream())
    torch.cuda.synchronize()
    got = torch.cat([t.cpu() for t in ranks.output()], 1)
    ranks.finish()
    return full.double().cpu().numpy(), got


def check(x, p, dtype, rules, **layout):
    x, got = run(x, p, dtype, rules, **layout)
    want, off = exact(x, rules)
    size = np.abs(np.where(np.isfinite(want), want, 0.0))
    tol = HALF_STEP[dtype] * (size + off) + off + FLOOR[dtype]
    assert_within(got, torch.from_numpy(want), torch.from_numpy(tol), f"{dtype} p={p}")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("p,rows,vocab,history,bias,mask", [
    (1, 1, 1, 3, 2, True), (1, 3, 7, 20, 0, False), (3, 2, 2, 9, 3, True), (2, 5, 1000, 300, 40, True),
    (4, 6, 5003, 1000, 0, True), (8, 4, 32768, 0, 10, True), (8, 7, 32000, 2000, 300, True), (1, 2, 50021, 70, 5, False),
    (3, 9, 33, 1, 1, True), (16, 3, 1001, 64, 7, True), (64, 2, 4099, 128, 7, False), (5, 300, 9001, 40, 4, True)])
def test_rules_match_the_definition(dtype, p, rows, vocab, history, bias, mask):
    x = rng(rows + vocab).normal(0, 4, (rows, vocab))
    check(x, p, dtype, make_rules(rows, vocab, 5, history, bias, mask))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [dict(ld=2051), dict(ld=2056, offset=8), dict(offset=1), dict(offset=[0, 3, 1, 2]),
                                    dict(offset=3, out_offset=1), dict(ld=2049, in_place=True), dict(in_place=True, offset=5)])
def test_strides_offsets_and_in_place(dtype, layout):
    rows, vocab = 6, 8190
    x = rng(1).normal(0, 4, (rows, vocab))
    check(x, 4, dtype, make_rules(rows, vocab, 9, 200, 30, True), **layout)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_large_batches_take_the_wide_slices(dtype):
    rows, vocab = 40, 150001
    x = rng(2).normal(0, 4, (rows, vocab))
    check(x, 2, dtype, make_rules(rows, vocab, 3, 500, 20, True))
    check(x, 2, dtype, make_rules(rows, vocab, 4, 500, 20, True), in_place=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,rows,vocab,history,bias,layout", [
    (2, 40, 150001, 3000, 20, {}), (8, 40, 131072, 9000, 700, {}), (3, 60, 100003, 1024, 1, dict(offset=3)),
    (1, 30, 200001, 40000, 5, dict(in_place=True)), (16, 60, 90011, 5000, 64, dict(offset=[0, 1] * 8)), (5, 400, 16000, 2000, 0, {})])
def test_long_histories_of_large_batches(dtype, p, rows, vocab, history, bias, layout):
    x = rng(vocab).normal(0, 4, (rows, vocab))
    check(x, p, dtype, make_rules(rows, vocab, 7, history, bias, True), **layout)


@pytest.mark.parametrize("history", [16383, 16384, 32768, 70000])
def test_a_token_repeated_through_a_long_history(history):
    """Counts around what a 16-bit counter holds, beside a neighbour that must not feel them."""
    a = make_rules(2, 300, 4).h
    a["history"] = np.full((2, history), 7, dtype=np.int32)
    a["history"][1, ::2] = 6
    a["prompt_len"] = np.array([0, 5], dtype=np.int32)
    check(rng(6).normal(0, 4, (2, 300)), 1, "f32", Rules(**a))


def test_each_rule_alone_and_none():
    rows, vocab = 5, 700
    x = rng(3).normal(0, 4, (rows, vocab))
    every = make_rules(rows, vocab, 8, 100, 9, True).h
    history = {k: every[k] for k in ("history", "history_len", "prompt_len")}
    for arrays in ({}, {**history}, {**history, "repetition": every["repetition"]}, {**history, "presence": every["presence"]},
                   {**history, "frequency": every["frequency"]}, {"history": every["history"], "frequency": every["frequency"]},
                   {k: every[k] for k in ("bias_offsets", "bias_tokens", "bias_values")}, {"mask": every["mask"]},
                   {"repetition": every["repetition"]}):
        check(x, 2, "bf16", Rules(**arrays))


def test_what_no_rule_touches_keeps_its_bits():
    vocab = 4096
    special = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min, 1e-40],
                           dtype=torch.bfloat16)
    full = special.repeat(vocab // 6 + 1)[:vocab].repeat(3, 1).cuda()
    rules = make_rules(3, vocab, 2)
    ranks = Ranks(shards(full, 2), "bf16")
    ccl.ccl_logit_rules(ranks.comm, "bf16", 3, vocab, rules.s, stream=stream())
    torch.cuda.synchronize()
    got = torch.cat([b.view for b in ranks.outs], 1)
    assert torch.equal(got.view(torch.int16), full.view(torch.int16))
    ranks.finish()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinite_and_lowest_logits(dtype):
    """NaN where the mask forbids is gone; -inf and the type's lowest value stay what the formula makes of them."""
    rows, vocab = 4, 999
    x = rng(4).normal(0, 4, (rows, vocab))
    x[0, ::3] = -np.inf
    x[1, ::3] = float(torch.finfo(TORCH[dtype]).min)
    x[2, ::3] = np.inf
    a = make_rules(rows, vocab, 6, 400, 0, True).h
    a["mask_index"] = np.arange(rows, dtype=np.int32)
    a["mask"][3] = 0                                  # nothing is allowed
    x[3] = np.nan
    a["repetition"][:] = 0.9                          # the lowest value divided or multiplied stays finite in fp32
    a["repetition"][1] = 1.0
    a["frequency"][:] = 0.0
    check(x, 3, dtype, Rules(**a))


def test_bias_entries_of_one_token_add_in_list_order():
    """(big + small) - big: another order gives another sum."""
    tokens = np.array([5, 9, 5, 5, 9, 5] * 20, dtype=np.int32)
    values = np.array([1e8, 1.0, 3.0, -1e8, 0.25, 1.0] * 20, dtype=np.float32)
    want = np.zeros(16, dtype=np.float32)
    for t, v in zip(tokens, values):
        want[t] = np.float32(want[t] + v)
    rules = Rules(bias_offsets=np.array([0, len(tokens)], dtype=np.int32), bias_tokens=tokens, bias_values=values)
    ranks = Ranks(shards(torch.zeros(1, 16, device="cuda"), 1), "f32")
    ccl.ccl_logit_rules(ranks.comm, "f32", 1, 16, rules.s, stream=stream())
    torch.cuda.synchronize()
    assert np.array_equal(ranks.outs[0].view.cpu().numpy()[0], want)
    ranks.finish()


@pytest.mark.parametrize("entries", [600, 9000])
def test_more_bias_entries_than_a_slice_keeps(entries):
    """All of one row's entries in one slice, some tokens many times; the other row has few."""
    g = rng(8)
    rows, vocab = 2, 4000
    a = {"bias_offsets": np.array([0, entries, entries + 3], dtype=np.int32),
         "bias_tokens": g.integers(100, 400, entries + 3).astype(np.int32),
         "bias_values": g.normal(0, 1, entries + 3).astype(np.float32)}
    check(g.normal(0, 4, (rows, vocab)), 1, "f32", Rules(**a))
    check(g.normal(0, 4, (rows, vocab)), 2, "bf16", Rules(**a), offset=3)


def test_bad_offsets_and_lengths_are_held_to_the_lists():
    rows, vocab = 4, 64
    x = rng(5).normal(0, 1, (rows, vocab))
    a = make_rules(rows, vocab, 1, 50, 8).h
    a["bias_offsets"] = np.array([-7, 3, 1, 2 ** 31 - 1, -5], dtype=np.int32)
    a["history_len"] = np.array([2 ** 31 - 1, -2 ** 31, 0, 10], dtype=np.int32)
    a["prompt_len"] = np.array([5, 0, 2 ** 31 - 1, -2 ** 31], dtype=np.int32)
    check(x, 2, "f32", Rules(**a))


def test_no_rows():
    ranks = Ranks([torch.zeros(1, 8, device="cuda")], "f32")
    ccl.ccl_logit_rules(ranks.comm, "f32", 0, 8, Rules().s, stream=stream())
    ranks.finish(wrote=False)


def test_another_stream_and_a_graph():
    rows, vocab, p = 6, 5000, 2
    x = torch.from_numpy(rng(7).normal(0, 4, (rows, vocab))).cuda().bfloat16()
    rules = make_rules(rows, vocab, 3, 200, 20, True)
    ranks = Ranks(shards(x, p), "bf16")
    call = lambda: ccl.ccl_logit_rules(ranks.comm, "bf16", rows, vocab, rules.s, stream=stream())
    call()
    torch.cuda.synchronize()
    want = [b.view.clone() for b in ranks.outs]
    for b in ranks.outs:
        b.view.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(b.view.view(torch.int16), w.view(torch.int16)) for b, w in zip(ranks.outs, want))
    ranks.finish()


def test_offsets_beyond_32_bits():
    vocab, rows = 32768, 2 ** 32 // 32768 + 5
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    y = torch.full((rows, vocab), 7.0, dtype=torch.bfloat16, device="cuda")
    history = torch.full((rows, 1), 5, dtype=torch.int32, device="cuda")
    history[-1, 0] = vocab - 1
    presence = torch.full((rows,), 0.5, device="cuda")
    mask = torch.full((1, vocab // 32), -1, dtype=torch.int32, device="cuda")
    mask[0, -1] = ~(1 << 30)
    index = torch.zeros(rows, dtype=torch.int32, device="cuda")
    rules = ccl.LogitRules(presence=presence.data_ptr(), history=history.data_ptr(), history_ld=1, mask=mask.data_ptr(), mask_rows=1,
                           mask_ld=vocab // 32, mask_index=index.data_ptr())
    want = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    want[:, 5] = -0.5
    want[-1, 5], want[-1, -1] = 0.0, -0.5
    want[:, vocab - 2] = -float("inf")
    for out in (y, x):                      # out of place, then in place
        comm = ccl.ccl_comm_create(1, [x.data_ptr()])
        ccl.ccl_comm_set_outputs(comm, [out.data_ptr()])
        ccl.ccl_logit_rules(comm, "bf16", rows, vocab, rules, stream=stream())
        ccl.ccl_comm_check(comm)
        ccl.ccl_comm_destroy(comm)
        assert torch.equal(out, want)

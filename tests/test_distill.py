"""GPU tests of ccl_distill_topk against a plain fp64 evaluation.

Tolerances.  u = 2^-24.  A probability is the product of at most two
exponentials of arguments up to R = (max - min of the finite logits) / T in
size (each argument meets three roundings, so 3 u R, and 2^x is good to 4 u)
over a sum of at most 128 additions in a row: (6 R + 3 R + 8 + 4 + 128 + 4) u,
taken as (10 R + 160) u relative.  The teacher's q: (10 Rt + k + 16) u.  The
loss is T^2 times sums of q (log q - log p), whose logarithms are off by the
same amounts absolutely."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import FLOOR, HALF_STEP, TORCH, U32, Ranks, assert_within, ptr, rng, shards, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def exact(z, ids, t, T, weight):
    """loss, gradient, statistics and the tolerances of loss and gradient (before its last rounding), fp64."""
    rows, vocab = z.shape
    ok = (ids >= 0) & (ids < vocab) & (t != -np.inf)
    at = np.where(ok, ids, 0)
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        m0 = np.where(m == -np.inf, 0.0, m)
        e = np.exp((z - m0) / T)
        total = e.sum(1, keepdims=True)
        p = np.where(total == 0, 0.0, e / total)
        ls = np.log(total)
        tm = np.where(ok, t, -np.inf).max(1, keepdims=True)
        taught = tm != -np.inf
        u = np.where(ok, (t - np.where(taught, tm, 0.0)) / T, -np.inf)
        w = np.exp(u)
        ts = w.sum(1, keepdims=True)
        q = np.where(taught, w / ts, 0.0)
        lq = np.where(q > 0, u - np.log(ts), 0.0)
        lp = np.where(total == 0, -np.inf, (np.take_along_axis(z, at, 1) - m0) / T - ls)
        loss = T * T * np.where(q > 0, q * (lq - np.where(q > 0, lp, 0.0)), 0.0).sum(1)
        share = np.zeros_like(z)
        for i in range(rows):
            np.add.at(share[i], at[i], q[i])
        factor = (np.ones(rows) if weight is None else weight)[:, None] * T
        grad = np.where(taught, factor * (p - share), 0.0)
        finite = np.isfinite(z)
        low = np.where(finite, z, np.inf).min(1, keepdims=True)
        # what lies 100 T below the maximum has no weight in fp32 either
        R = np.where(finite.any(1, keepdims=True), np.minimum((m0 - low) / T, 100.0), 0.0)
        Rt = np.where(taught, np.minimum(-np.where(np.isfinite(u), u, 0.0).min(1, keepdims=True), 100.0), 0.0)
        k = ids.shape[1]
        dp, dq = (10 * R + 160) * U32, (10 * Rt + k + 16) * U32
        dgrad = np.abs(factor) * (p * dp + share * dq + (p + share) * 4 * U32)
        far = np.where(np.isfinite(lp), np.abs(lp), 0.0).max(1, keepdims=True)
        dloss = T * T * (dp + dq + (dq + 8 * U32) * (far + Rt + np.log(k + 1.0)) + 4 * U32 * far)
        # a loss whose terms leave fp32's range
        loss = np.where(loss > 3.4028235e38, np.inf, loss)
    return loss, grad, m[:, 0], ls[:, 0], dloss[:, 0], dgrad, dp[:, 0]


def teacher(rows, vocab, k, seed, ragged=True):
    g = rng(seed)
    ids = np.stack([g.permutation(max(vocab, k))[:k] for _ in range(rows)]).astype(np.int32)   # some past the vocabulary
    if ragged:
        ids[g.random(ids.shape) < 0.1] = -1
        if k > 3:
            ids[:, 3] = ids[:, 0]                     # one token twice
            ids[0, 1:] = ids[0, 0]                    # and one k times
        if rows > 2:
            ids[2] = -1                               # a row without a teacher
    t = g.normal(0, 3, ids.shape)
    t[:, k // 2] = np.where(g.random(rows) < 0.3, -np.inf, t[:, k // 2])
    return ids, t


def check(z, ids, t, T, p, dtype, steps="both", weight=None, teacher_dtype="f32", keep_stats=True, **layout):
    rows, vocab = z.shape
    full = torch.from_numpy(z).cuda().to(TORCH[dtype])
    td = torch.from_numpy(t).cuda().to(TORCH[teacher_dtype])
    ids_d = torch.from_numpy(ids).cuda()
    w = None if weight is None else torch.from_numpy(weight).float().cuda()
    z64, t64 = full.double().cpu().numpy(), td.double().cpu().numpy()
    loss, grad, m, ls, dloss, dgrad, dp = exact(z64, ids, t64, T, None if w is None else w.double().cpu().numpy())
    ranks = Ranks(shards(full, p), dtype, **layout)
    got = torch.full((rows + 2,), float("nan"), device="cuda")
    stats = torch.full((rows + 2, 2), float("nan"), device="cuda")
    args = dict(teacher_dtype=teacher_dtype, temperature=T, row_weight=ptr(w), loss=got[1:].data_ptr(),
                stats=stats[1:].data_ptr() if keep_stats else 0, ld=layout.get("ld", 0), stream=stream())
    for s in {"both": ["both"], "forward": ["forward"], "each": ["forward", "backward"]}[steps]:
        ccl.ccl_distill_topk(ranks.comm, dtype, s, rows, vocab, ids.shape[1], ids_d.data_ptr(), td.data_ptr(), **args)
    torch.cuda.synchronize()
    assert_within(got[1:-1], torch.from_numpy(loss), torch.from_numpy(dloss + 2 * U32 * np.abs(np.where(np.isfinite(loss), loss, 0))), "loss")
    if keep_stats:
        assert_within(stats[1:-1, 0], torch.from_numpy(m), 0.0, "maximum")
        assert_within(stats[1:-1, 1], torch.from_numpy(ls), torch.from_numpy(dp + 4 * U32 * np.abs(np.where(np.isfinite(ls), ls, 0))), "log-sum")
    assert bool(torch.isnan(got[[0, -1]]).all()) and bool(torch.isnan(stats[[0, -1]]).all())
    if steps != "forward":
        out = torch.cat([x.cpu() for x in ranks.output()], 1)
        if steps == "each":      # through the stored statistics: their rounding counts too
            dgrad = dgrad + np.abs(grad + dgrad) * 4 * U32 * (2 + np.abs(np.where(np.isfinite(ls), ls, 0)))[:, None]
        tol = dgrad + HALF_STEP[dtype] * (np.abs(grad) + dgrad) + FLOOR[dtype]
        assert_within(out, torch.from_numpy(grad), torch.from_numpy(tol), f"gradient {dtype} p={p} {steps}")
    ranks.finish(wrote=steps != "forward")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("steps", ["both", "forward", "each"])
@pytest.mark.parametrize("p,rows,vocab,k,T", [
    (1, 1, 1, 1, 1.0), (1, 3, 7, 5, 2.0), (2, 4, 1000, 20, 1.0), (3, 5, 5003, 17, 0.5), (8, 4, 32768, 64, 2.0),
    (3, 200, 33, 4, 1.5), (16, 3, 2051, 8, 1.0), (64, 2, 4099, 100, 3.0), (8, 3, 5, 3, 1.0), (1, 6, 50021, 1024, 2.0),
    (2, 9, 9001, 65, 1.0), (4, 5, 12007, 129, 2.0), (2, 4, 40009, 700, 1.0), (9, 40, 6001, 33, 1.0), (33, 3, 7001, 80, 1.0)])
def test_matches_the_definition(dtype, steps, p, rows, vocab, k, T):
    g = rng(rows + vocab)
    ids, t = teacher(rows, vocab, k, 3)
    check(g.normal(0, 3, (rows, vocab)), ids, t, T, p, dtype, steps, weight=g.normal(0, 1, rows))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [dict(ld=2051), dict(ld=2056, offset=8), dict(offset=1), dict(offset=[0, 3, 1, 2]),
                                    dict(offset=3, out_offset=1), dict(ld=2049, in_place=True), dict(in_place=True, offset=5)])
@pytest.mark.parametrize("steps", ["both", "each"])
def test_strides_offsets_and_in_place(dtype, layout, steps):
    rows, vocab = 5, 8190
    ids, t = teacher(rows, vocab, 30, 4)
    check(rng(1).normal(0, 3, (rows, vocab)), ids, t, 1.0, 4, dtype, steps, **layout)


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 3, 300001), ("f32", 2, 270000), ("f16", 170, 140003), ("f32", 60, 131072),
                                              ("bf16", 400, 9000), ("f32", 170, 3001)])
@pytest.mark.parametrize("in_place", [False, True])
def test_vocabularies_below_and_beyond_what_a_cluster_keeps(dtype, rows, vocab, in_place):
    ids, t = teacher(rows, vocab, 16, 6)
    check(rng(2).normal(0, 3, (rows, vocab)), ids, t, 2.0, 2, dtype, "both", in_place=in_place)


@pytest.mark.parametrize("teacher_dtype", ["bf16", "f16", "f32"])
def test_teacher_types_and_optional_arrays(teacher_dtype):
    ids, t = teacher(4, 500, 12, 7)
    z = rng(3).normal(0, 3, (4, 500))
    check(z, ids, t, 1.0, 2, "bf16", "both", teacher_dtype=teacher_dtype, keep_stats=False)
    check(z, ids, t, 1.0, 2, "f32", "forward", teacher_dtype=teacher_dtype, keep_stats=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("steps", ["both", "each"])
@pytest.mark.parametrize("rows_like", [1, 40])
def test_masked_logits(dtype, steps, rows_like):
    """-inf and the type's lowest value in parts of a row, in whole parts of the ranks, and in all of it."""
    vocab, k = 40000, 6
    low = float(torch.finfo(TORCH[dtype]).min)
    g = rng(8)
    z = g.normal(0, 3, (8, vocab))
    ids, t = teacher(8, vocab, k, 9, ragged=False)
    z[0, ::2] = -np.inf
    z[1, ::2] = low
    z[2, : vocab // 2] = -np.inf                   # the first rank has nothing
    z[3, 1:] = -np.inf                             # one token is left
    z[4] = -np.inf                                 # none is
    z[5] = low                                     # a row of the lowest value: uniform
    z[6] -= 500.0                                  # far below zero, beside threads that hold -inf only
    z[6, 100:] = -np.inf
    z[7] += 300.0
    for i in (0, 2, 6):                            # the teacher keeps to what is left ...
        left = np.flatnonzero(z[i] != -np.inf)
        ids[i] = g.choice(left, k, replace=False)
    ids[3] = -1
    ids[3, 0] = 0
    t[t == -np.inf] = 0.0
    if rows_like > 1:
        z, ids, t = (np.tile(x, (rows_like, 1)) for x in (z, ids, t))
    check(z, ids, t, 1.0, 2, dtype, steps)
    check(z, ids, t, 0.25, 2, dtype, steps)        # 1 / T scales the lowest value beyond fp32


def test_the_teacher_insists_on_a_masked_token():
    """... or does not: the loss is infinite, the gradient finite."""
    z = rng(10).normal(0, 1, (3, 100))
    z[:, 50:] = -np.inf
    ids = np.array([[60, 3], [60, 61], [3, 4]], dtype=np.int32)
    t = np.array([[1.0, 2.0], [0.0, 0.0], [0.0, -np.inf]])
    check(z, ids, t, 1.0, 2, "f32", "both")


def test_nan_and_plus_infinity_reach_their_row_alone():
    z = rng(11).normal(0, 1, (3, 1000)).astype(np.float32)
    z[0, 7], z[2, 990] = np.nan, np.inf
    full = torch.from_numpy(z).cuda()
    ids = torch.tensor([[1, 2], [3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    t = torch.zeros(3, 2, device="cuda")
    loss = torch.empty(3, device="cuda")
    ranks = Ranks(shards(full, 2), "f32")
    ccl.ccl_distill_topk(ranks.comm, "f32", "both", 3, 1000, 2, ids.data_ptr(), t.data_ptr(), loss=loss.data_ptr(), stream=stream())
    out = torch.cat(ranks.output(), 1)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(loss), torch.tensor([True, False, True], device="cuda"))
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all()) and bool(torch.isnan(out[2]).all())
    ccl.ccl_comm_destroy(ranks.comm)


def test_gradient_against_differences():
    """The kernel's fp32 gradient against central differences of the fp64 loss: the difference quotient's own error is
    h^2 / 6 times a third derivative (at most 2 / T, of probabilities) plus 2^-52 of the loss over h."""
    rows, vocab, T, h = 3, 40, 1.5, 1e-3
    z = rng(12).normal(0, 2, (rows, vocab)).astype(np.float32).astype(np.float64)
    ids, t = teacher(rows, vocab, 5, 13)
    t = t.astype(np.float32).astype(np.float64)
    weight = np.array([0.5, 2.0, 1.0])
    slope = np.zeros_like(z)
    for v in range(vocab):
        up, down = z.copy(), z.copy()
        up[:, v] += h
        down[:, v] -= h
        slope[:, v] = (exact(up, ids, t, T, weight)[0] - exact(down, ids, t, T, weight)[0]) / (2 * h) * weight
    _, grad, _, _, _, dgrad, _ = exact(z, ids, t, T, weight)
    ranks = Ranks(shards(torch.from_numpy(z).cuda().float(), 3), "f32")
    loss = torch.empty(rows, device="cuda")
    keep = [torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda().float(), torch.from_numpy(weight).cuda().float()]
    ccl.ccl_distill_topk(ranks.comm, "f32", "both", rows, vocab, 5, *(x.data_ptr() for x in keep[:2]), temperature=T,
                         row_weight=keep[2].data_ptr(), loss=loss.data_ptr(), stream=stream())
    out = torch.cat(ranks.output(), 1)
    assert_within(out, torch.from_numpy(slope), torch.from_numpy(dgrad + 1e-6 * 2.0 + 1e-11), "difference quotient")
    ranks.finish()


def test_same_bits_again_on_another_stream_and_in_a_graph():
    rows, vocab, p, k = 300, 20011, 3, 40
    ids, t = teacher(rows, vocab, k, 14)
    full = torch.from_numpy(rng(14).normal(0, 3, (rows, vocab))).cuda().bfloat16()
    ids, t = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda().float()
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    ranks = Ranks(shards(full, p), "bf16")

    def call():
        ccl.ccl_distill_topk(ranks.comm, "bf16", "both", rows, vocab, k, ids.data_ptr(), t.data_ptr(), temperature=2.0,
                             loss=loss.data_ptr(), stats=stats.data_ptr(), stream=stream())

    def result():
        torch.cuda.synchronize()
        r = [b.view.clone().view(torch.int16) for b in ranks.outs] + [loss.clone().view(torch.int32), stats.clone().view(torch.int32)]
        for x in [b.view for b in ranks.outs] + [loss, stats]:
            x.zero_()
        torch.cuda.synchronize()
        return r

    call()
    want = result()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    assert all(torch.equal(a, b) for a, b in zip(result(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(result(), want))
    ranks.finish()


def test_offsets_beyond_32_bits():
    """More than 2^32 elements in one rank's buffer, in place; the last rows are checked."""
    rows, vocab, k, dtype = 33000, 131072, 8, "bf16"
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    tail = torch.from_numpy(rng(15).normal(0, 3, (4, vocab))).cuda().bfloat16()
    z[-4:] = tail
    ids, t = teacher(4, vocab, k, 16)
    ids_d = torch.full((rows, k), -1, dtype=torch.int32, device="cuda")
    t_d = torch.zeros(rows, k, device="cuda")
    ids_d[-4:], t_d[-4:] = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda().float()
    loss = torch.empty(rows, device="cuda")
    comm = ccl.ccl_comm_create(1, [z.data_ptr()])
    ccl.ccl_distill_topk(comm, dtype, "both", rows, vocab, k, ids_d.data_ptr(), t_d.data_ptr(), loss=loss.data_ptr(), stream=stream())
    torch.cuda.synchronize()
    want, grad, _, _, dloss, dgrad, _ = exact(tail.double().cpu().numpy(), ids, t_d[-4:].double().cpu().numpy(), 1.0, None)
    assert_within(loss[-4:], torch.from_numpy(want), torch.from_numpy(dloss + 2 * U32 * want), "loss")
    tol = dgrad + HALF_STEP[dtype] * (np.abs(grad) + dgrad) + FLOOR[dtype]
    assert_within(z[-4:], torch.from_numpy(grad), torch.from_numpy(tol), "gradient")
    assert bool((loss[:-4] == 0).all()) and bool((z[:100] == 0).all()) and bool((z[-104:-4] == 0).all())
    ccl.ccl_comm_destroy(comm)


@pytest.mark.parametrize("steps", ["forward", "both", "backward"])
def test_a_wait_that_runs_out_is_reported(steps):
    """A load is withheld (the test hook): the call ends, ccl_comm_check reports it, and the next call is whole."""
    rows, vocab = 700, 3000
    ids, t = teacher(rows, vocab, 4, 20)
    full = torch.from_numpy(rng(20).normal(0, 3, (rows, vocab))).cuda().bfloat16()
    ids_d, t_d = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda().float()
    loss, stats = torch.empty(rows, device="cuda"), torch.zeros(rows, 2, device="cuda")
    ranks = Ranks(shards(full, 3), "bf16")

    def call():
        ccl.ccl_distill_topk(ranks.comm, "bf16", steps, rows, vocab, 4, ids_d.data_ptr(), t_d.data_ptr(), loss=loss.data_ptr(),
                             stats=stats.data_ptr(), stream=stream())

    ccl.ccl_comm_set_debug(ranks.comm, 2_000_000, 1)
    call()
    with pytest.raises(ccl.CclError) as e:
        ccl.ccl_comm_check(ranks.comm)
    assert e.value.status == ccl.CCL_ERR_TIMEOUT
    ccl.ccl_comm_set_debug(ranks.comm, 0, 0)
    call()
    ccl.ccl_comm_check(ranks.comm)
    if steps != "backward":
        want, *_, dloss, _, _ = exact(full.double().cpu().numpy(), ids, t_d.double().cpu().numpy(), 1.0, None)
        assert_within(loss, torch.from_numpy(want), torch.from_numpy(dloss + 2 * U32 * np.abs(want)), "loss")
    ccl.ccl_comm_destroy(ranks.comm)


def test_no_rows():
    ranks = Ranks([torch.zeros(1, 8, device="cuda")], "f32")
    one = torch.zeros(8, device="cuda")
    ccl.ccl_distill_topk(ranks.comm, "f32", "both", 0, 8, 2, one.data_ptr(), one[4:].data_ptr(), loss=one[6:].data_ptr(), stream=stream())
    ranks.finish(wrote=False)


@pytest.mark.parametrize("p,rows,vocab,dtype,layout", [
    (3, 330, 5003, "bf16", {}), (8, 310, 8000, "f16", {}), (8, 160, 32000, "bf16", dict(in_place=True)), (5, 400, 1003, "f32", {}),
    (7, 320, 61, "bf16", {}), (4, 310, 9001, "f32", dict(offset=[0, 3, 1, 2])), (3, 60, 100003, "bf16", {}),
    (8, 70, 80725, "bf16", dict(offset=3, out_offset=1)), (8, 75, 80725, "bf16", dict(in_place=True)),
    (6, 320, 2047, "f16", dict(ld=400, in_place=True)), (2, 320, 20, "f32", {}), (12, 80, 40009, "f32", {}), (20, 330, 1201, "bf16", {})])
@pytest.mark.parametrize("steps", ["both", "forward", "each"])
def test_pieces_over_several_shards(p, rows, vocab, dtype, layout, steps):
    """Rows enough for every SM: then a piece may end inside one shard and go on in the next."""
    g = rng(rows * p)
    ids, t = teacher(rows, vocab, min(40, vocab), 8)
    edge = np.cumsum([0] + [vocab // p + (r < vocab % p) for r in range(p)])
    ids[1::3, 0], ids[2::3, 1] = edge[1] - 1, edge[1] % vocab      # on both sides of a bound
    check(g.normal(0, 3, (rows, vocab)), ids, t, 1.5, p, dtype, steps, weight=g.normal(0, 1, rows), **layout)

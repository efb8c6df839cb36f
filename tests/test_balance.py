"""GPU tests of ccl_balance_loss against a plain fp64 evaluation.

Tolerances.  u = 2^-24, R = max - min of a row's finite logits, E experts.  A
probability is an exponential (3 u R + 4 u) over a sum of at most 64 additions
in a row, each lane's included: dp = (6 R + 80) u relative (E above 1024: one
more addition per 32 experts).  d_e = a_e - mean(a) is rounded once, u |d_e|.
The row's sum of p d is off by at most max|d| (dp + 80 u); the gradient by
|dloss| p (max|d| (3 dp + 160 u)).  The loss adds the rows' sums in fp32 per
thread, at most n of them: n u of their total magnitude."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import FLOOR, HALF_STEP, TORCH, U32, Ranks, assert_within, ptr, rng, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def exact(xs, ids, valid, coef, dloss):
    """loss, gradients, counts, tokens and the tolerances of loss and gradients, fp64, by the formula."""
    p, (rows, E), k = len(xs), xs[0].shape, ids[0].shape[1]
    keep = [np.ones(rows, bool) if valid is None else valid[r] != 0 for r in range(p)]
    counts = np.stack([np.bincount(i[v][(i[v] >= 0) & (i[v] < E)], minlength=E) for i, v in zip(ids, keep)])
    tokens = np.array([int(v.sum()) for v in keep])
    n = tokens.sum()
    total = counts.sum(0)
    scale = coef * E / (k * float(n) ** 2) if n else 0.0
    a, d = total * scale, (total - total.mean()) * scale    # the gradient is one of differences: equal counts give 0 exactly
    top = np.abs(d).max()
    loss, off, grads, tols = 0.0, 0.0, [], []
    for x, v in zip(xs, keep):
        with np.errstate(all="ignore"):
            m = x.max(1, keepdims=True)
            m = np.where(m == -np.inf, 0.0, m)
            e = np.exp(x - m)
            s = e.sum(1, keepdims=True)
            prob = np.where(s == 0, 0.0, e / s)
            prob = np.where(v[:, None], prob, 0.0)
            low = np.where(np.isfinite(x), x, np.inf).min(1, keepdims=True)
            R = np.where(np.isfinite(low), np.minimum(m - low, 100.0), 0.0)
        dp = (6 * R + 80 + E // 32) * U32
        loss += (prob * a).sum()
        off += (top * (dp + 80 * U32))[v].sum()
        grads.append(dloss * prob * (d - (prob * d).sum(1, keepdims=True)))
        tols.append(abs(dloss) * prob * top * (3 * dp + 160 * U32))
    # each thread adds at most rows of the largest sum; the conversions to fp32 at the end
    off += rows * n * U32 * top + 8 * U32 * abs(loss)
    return loss, grads, counts, tokens, off, tols


def choices(rows, E, k, p, seed, drop=0.05):
    g = rng(seed)
    ids = [np.stack([g.permutation(E)[:k] for _ in range(rows)]).astype(np.int32).reshape(rows, k) for _ in range(p)]
    for i in ids:
        i[g.random(i.shape) < drop] = -1
        i[g.random(i.shape) < drop] = E
        i[:, 0] = np.where(g.random(rows) < 0.5, 0, i[:, 0])        # a favourite
    return ids


def check(xs, ids, dtype, steps="both", valid=None, coef=0.01, dloss=512.0, repeat=1, **layout):
    p, (rows, E), k = len(xs), xs[0].shape, ids[0].shape[1]
    parts = [torch.from_numpy(x).cuda().to(TORCH[dtype]) for x in xs]
    x64 = [t.double().cpu().numpy() for t in parts]
    loss, grads, counts, tokens, off, tols = exact(x64, ids, valid, float(np.float32(coef)), 1.0 if dloss is None else dloss)
    ranks = Ranks(parts, dtype, **layout)
    ids_d = [torch.from_numpy(i).cuda() for i in ids]
    v_d = None if valid is None else [torch.from_numpy(v).cuda() for v in valid]
    up = None if dloss is None else torch.tensor([dloss], device="cuda")
    cnt = torch.full((p * E + 2,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((p + 2,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((3,), float("nan"), device="cuda")
    for s in {"both": ["both"], "forward": ["forward"], "each": ["forward", "backward"]}[steps] * repeat:
        ccl.ccl_balance_loss(ranks.comm, dtype, s, rows, E, k, None if s == "backward" else [i.data_ptr() for i in ids_d],
                             None if v_d is None else [v.data_ptr() for v in v_d], coef, ptr(up), cnt[1:].data_ptr(),
                             tok[1:].data_ptr(), 0 if s == "backward" else out[1:].data_ptr(), stream=stream())
    torch.cuda.synchronize()
    assert np.array_equal(cnt[1:-1].cpu().numpy().reshape(p, E), counts)
    assert np.array_equal(tok[1:-1].cpu().numpy(), tokens)
    assert bool((cnt[[0, -1]] == -7).all()) and bool((tok[[0, -1]] == -7).all()) and bool(torch.isnan(out[[0, 2]]).all())
    assert_within(out[1:2], torch.tensor([loss]), off, "loss")
    if steps != "forward":
        for r, got in enumerate(ranks.output()):
            tol = tols[r] + HALF_STEP[dtype] * (np.abs(grads[r]) + tols[r]) + FLOOR[dtype]
            assert_within(got, torch.from_numpy(grads[r]), torch.from_numpy(tol), f"gradient of rank {r}")
    ranks.finish(wrote=steps != "forward")


def padding(rows, p, seed):
    g = rng(seed)
    v = [(g.random(rows) < 0.7).astype(np.uint8) * g.integers(1, 255, rows).astype(np.uint8) for _ in range(p)]
    v[-1][:] = 0                                     # a rank of padding alone
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("steps", ["both", "forward", "each"])
@pytest.mark.parametrize("p,rows,E,k", [
    (1, 1, 1, 1), (1, 1, 8, 2), (2, 5, 8, 1), (3, 33, 16, 4), (8, 64, 64, 6), (2, 1000, 60, 4), (4, 300, 61, 3),
    (2, 257, 128, 8), (3, 700, 256, 8), (16, 40, 384, 8), (1, 90, 512, 2), (2, 50, 640, 8), (1, 70, 1024, 4), (2, 9, 1500, 8),
    (1, 6, 4096, 16), (64, 3, 32, 2), (8, 2100, 96, 1), (5, 17, 7, 7)])
def test_matches_the_definition(dtype, steps, p, rows, E, k):
    g = rng(rows * E)
    xs = [g.normal(0, 2, (rows, E)) for _ in range(p)]
    check(xs, choices(rows, E, k, p, 1), dtype, steps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,rows,E,k", [(2, 100, 64, 4), (3, 5000, 128, 6), (4, 77, 30, 2), (2, 3000, 2, 1)])
def test_padding_rows(dtype, p, rows, E, k):
    g = rng(3)
    xs = [g.normal(0, 2, (rows, E)) for _ in range(p)]
    valid = padding(rows, p, 4)
    for x, v in zip(xs, valid):
        x[v == 0] = np.nan                           # what padding holds does not matter
        x[v == 0, :1] = np.inf
    for steps in ("both", "forward", "each"):
        check(xs, choices(rows, E, k, p, 2), dtype, steps, valid)


@pytest.mark.parametrize("layout", [dict(offset=1), dict(offset=3, out_offset=2), dict(in_place=True), dict(in_place=True, offset=1),
                                    dict(offset=0, out_offset=4)])
def test_offsets_and_in_place(layout):
    g = rng(5)
    xs = [g.normal(0, 2, (400, 64)) for _ in range(2)]
    check(xs, choices(400, 64, 4, 2, 6), "bf16", "both", **layout)
    check(xs, choices(400, 64, 4, 2, 6), "f32", "both", **layout)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E", [32, 33])
def test_masked_experts_and_rows(dtype, E):
    g = rng(7)
    x = g.normal(0, 2, (200, E))
    low = float(torch.finfo(TORCH[dtype]).min)
    x[::4, ::3] = -np.inf
    x[1::4, ::3] = low
    x[2] = -np.inf
    x[6] = low
    x[10, 1:] = -np.inf
    for steps in ("both", "each"):
        check([x, x[::-1].copy()], choices(200, E, 3, 2, 8), dtype, steps)


@pytest.mark.parametrize("rows", [0, 5])
def test_without_a_valid_row(rows):
    xs = [np.ones((rows, 16)), np.ones((rows, 16))]
    ids = choices(rows, 16, 2, 2, 1) if rows else [np.zeros((0, 2), np.int32)] * 2
    parts = [torch.from_numpy(x).cuda() .float() for x in xs]
    if rows:
        check(xs, ids, "f32", "each", [np.zeros(rows, np.uint8)] * 2)
        return
    one = torch.full((4,), 3.0, device="cuda")
    cnt, tok = torch.full((32,), 5, dtype=torch.int32, device="cuda"), torch.full((2,), 5, dtype=torch.int32, device="cuda")
    comm = ccl.ccl_comm_create(2, [one.data_ptr(), one.data_ptr() + 8])
    for steps in ("both", "backward"):
        ccl.ccl_balance_loss(comm, "f32", steps, 0, 16, 2, [one.data_ptr()] * 2, None, 0.1, 0, cnt.data_ptr(), tok.data_ptr(),
                             one[1:].data_ptr(), stream=stream())
    torch.cuda.synchronize()
    assert one.tolist() == [3.0, 0.0, 3.0, 3.0] and not cnt.any() and not tok.any()
    ccl.ccl_comm_destroy(comm)


def test_balanced_choices_leave_a_zero_gradient():
    """Equal counts: a_e is the mean for every expert, so the gradient is exactly 0 and the loss coef."""
    rows, E = 256, 16
    ids = [(np.arange(rows * 2, dtype=np.int32) % E).reshape(rows, 2)]
    x = rng(9).normal(0, 3, (rows, E))
    check([x], ids, "f32", "both", coef=0.5)
    parts = torch.from_numpy(x).cuda().float()
    ranks = Ranks([parts], "f32")
    ids_d = torch.from_numpy(ids[0]).cuda()
    cnt, tok, loss = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    ccl.ccl_balance_loss(ranks.comm, "f32", "both", rows, E, 2, [ids_d.data_ptr()], None, 0.5, 0, cnt.data_ptr(), tok.data_ptr(),
                         loss.data_ptr(), stream=stream())
    torch.cuda.synchronize()
    assert not bool(ranks.outs[0].view.any()) and abs(float(loss) - 0.5) <= 8 * U32
    ranks.finish()


def test_optional_upstream_gradient_and_calls_in_a_row():
    xs = [rng(10).normal(0, 2, (3000, 64)) for _ in range(2)]
    ids = choices(3000, 64, 6, 2, 11)
    check(xs, ids, "f32", "both", dloss=None, repeat=5)
    check([x[:20] for x in xs], [i[:20] for i in ids], "bf16", "each", repeat=5)


def test_gradient_against_differences():
    """The difference quotient of the fp64 loss: h^2 / 6 times a third derivative of softmaxes (below 1) times max a."""
    rows, E, k, h = 3, 6, 2, 1e-3
    g = rng(12)
    xs = [g.normal(0, 1, (rows, E)).astype(np.float32).astype(np.float64) for _ in range(2)]
    ids = choices(rows, E, k, 2, 13)
    coef, up = float(np.float32(0.3)), 8.0
    slope = [np.zeros((rows, E)) for _ in xs]
    for r in range(2):
        for t in range(rows):
            for e in range(E):
                both = []
                for sign in (h, -h):
                    moved = [x.copy() for x in xs]
                    moved[r][t, e] += sign
                    both.append(exact(moved, ids, None, coef, up)[0])
                slope[r][t, e] = up * (both[0] - both[1]) / (2 * h)
    _, grads, _, _, _, tols = exact(xs, ids, None, coef, up)
    parts = [torch.from_numpy(x).cuda().float() for x in xs]
    ranks = Ranks(parts, "f32")
    ids_d = [torch.from_numpy(i).cuda() for i in ids]
    cnt, tok = torch.empty(2 * E, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    loss, dl = torch.empty(1, device="cuda"), torch.tensor([up], device="cuda")
    ccl.ccl_balance_loss(ranks.comm, "f32", "both", rows, E, k, [i.data_ptr() for i in ids_d], None, coef, dl.data_ptr(),
                         cnt.data_ptr(), tok.data_ptr(), loss.data_ptr(), stream=stream())
    for got, want, tol in zip(ranks.output(), slope, tols):
        assert_within(got, torch.from_numpy(want), torch.from_numpy(tol + up * 0.3 * 1e-6 + 1e-11), "difference quotient")
    ranks.finish()


@pytest.mark.parametrize("rows", [50, 5000])
def test_same_bits_again_on_another_stream_and_in_a_graph(rows):
    E, k, p = 64, 4, 3
    parts = [torch.from_numpy(rng(r).normal(0, 2, (rows, E))).cuda().bfloat16() for r in range(p)]
    ids = [torch.from_numpy(i).cuda() for i in choices(rows, E, k, p, 14)]
    cnt, tok, loss = torch.empty(p * E, dtype=torch.int32, device="cuda"), torch.empty(p, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    ranks = Ranks(parts, "bf16")

    def call():
        ccl.ccl_balance_loss(ranks.comm, "bf16", "both", rows, E, k, [i.data_ptr() for i in ids], None, 0.01, 0, cnt.data_ptr(),
                             tok.data_ptr(), loss.data_ptr(), stream=stream())

    def result():
        torch.cuda.synchronize()
        r = [b.view.clone().view(torch.int16) for b in ranks.outs] + [cnt.clone(), tok.clone(), loss.clone().view(torch.int32)]
        for x in [b.view for b in ranks.outs] + [cnt, tok, loss]:
            x.zero_()
        torch.cuda.synchronize()
        return r

    call()
    want = result()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
        call()
    assert all(torch.equal(a, b) for a, b in zip(result(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(result(), want))
    ranks.finish()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E", [1, 3, 9, 15, 17, 31, 45, 100, 127, 130, 255, 259, 500, 511, 513, 700, 1023])
@pytest.mark.parametrize("layout", [dict(), dict(in_place=True, offset=1), dict(offset=[0, 1, 2], out_offset=3)])
def test_rows_that_are_no_aligned_groups(dtype, E, layout):
    g = rng(E)
    rows = 37 if E > 100 else 211
    xs = [g.normal(0, 2, (rows, E)) for _ in range(3)]
    valid = padding(rows, 3, E)
    for x, v in zip(xs, valid):
        x[v == 0] = np.nan
    check(xs, choices(rows, E, min(E, 3), 3, E), dtype, "both", valid, **layout)


@pytest.mark.parametrize("E,offset", [(64, 0), (61, 0), (64, 1)])
def test_offsets_beyond_32_bits(E, offset):
    rows, some = 2 ** 32 // E + 77, 5
    g = rng(E)
    tail = torch.from_numpy(g.normal(0, 2, (some, E))).cuda().bfloat16()
    x = torch.zeros(rows * E + offset, dtype=torch.bfloat16, device="cuda")
    x[-some * E:] = tail.view(-1)
    y = torch.full((rows * E + offset,), 7.0, dtype=torch.bfloat16, device="cuda")
    size = x.element_size() * offset
    counts, tokens = torch.from_numpy(g.integers(0, 1000, E).astype(np.int32)).cuda(), torch.tensor([1000], dtype=torch.int32, device="cuda")
    up = torch.tensor([4096.0], device="cuda")
    comm = ccl.ccl_comm_create(1, [x.data_ptr() + size])
    ccl.ccl_comm_set_outputs(comm, [y.data_ptr() + size])
    ccl.ccl_balance_loss(comm, "bf16", "backward", rows, E, 2, None, None, 1.0, up.data_ptr(), counts.data_ptr(),
                         tokens.data_ptr(), 0, stream=stream())
    ccl.ccl_comm_check(comm)
    ccl.ccl_comm_destroy(comm)
    c = counts.double().cpu()
    d = (c - c.mean()) * E / (2 * 1000.0 ** 2)
    z = torch.cat([torch.zeros(1, E), tail.double().cpu()])
    prob = z.softmax(1)
    want = 4096.0 * prob * (d - (prob * d).sum(1, keepdim=True))
    R = z.max(1, keepdim=True).values - z.min(1, keepdim=True).values
    tol = 4096.0 * prob * d.abs().max() * (3 * (6 * R + 80) + 160) * U32
    tol = tol + HALF_STEP["bf16"] * (want.abs() + tol) + FLOOR["bf16"]
    got = y[offset:].view(rows, E)
    assert_within(got[-some:], want[1:], tol[1:], "the last rows")
    for r in (0, 2 ** 31 // E, 2 ** 31 // E + 1, rows // 2, rows - some - 1):
        assert_within(got[r], want[0], tol[0], f"row {r}")

"""The operators around the layers of a model whose ranks' buffers one GPU
holds, as cases to measure: each in a plain form (elementary torch operations
in fp32) and as the calls a user makes.

  norm      AllReduce, residual and RMSNorm with an 8-bit (e4m3) output and
            its scales
  sort      a router's choices: the row of the expert's buffer for each, and
            where each expert's rows begin
  dispatch  tokens of all ranks to the buffers of their experts' ranks
  combine   the experts' rows back to the tokens, weighted and summed
  gradient  combine's gradient, of the experts' rows and of the weights
  clip      the global norm of many gradient tensors, and their clipping
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # a decode step of a small batch, block scales for the product that follows: latency
        {"name": "norm, decode step", "op": "norm", "dtype": "bf16", "p": 8, "rows": 8, "hidden": 7168, "group": 128},
        # a prompt's tokens, a scale for each
        {"name": "norm, prompt", "op": "norm", "dtype": "f16", "p": 4, "rows": 4000, "hidden": 8192, "group": 0},
        # the choices of one decode step: latency
        {"name": "sort, decode step", "op": "sort", "p": 8, "rows": 16, "experts": 256, "k": 8, "padding": False},
        # a training step of eight ranks, many small experts, padded sequences
        {"name": "sort, training step", "op": "sort", "p": 8, "rows": 16384, "experts": 256, "k": 8, "padding": True},
        # an odd width and odd counts, few ranks
        {"name": "dispatch, odd sizes", "op": "dispatch", "dtype": "f32", "p": 3, "rows": 1111, "hidden": 1001,
         "experts": 20, "k": 2, "weighted": False},
        # a prompt's tokens to the experts of eight ranks
        {"name": "dispatch, prompt", "op": "dispatch", "dtype": "bf16", "p": 8, "rows": 4096, "hidden": 7168,
         "experts": 256, "k": 8, "weighted": False},
        # a decode step's rows back to their tokens: latency
        {"name": "combine, decode step", "op": "combine", "dtype": "bf16", "p": 8, "rows": 16, "hidden": 7168,
         "experts": 256, "k": 8, "weighted": True},
        # a training step of four ranks
        {"name": "combine, training step", "op": "combine", "dtype": "f16", "p": 4, "rows": 8192, "hidden": 4096,
         "experts": 64, "k": 6, "weighted": True},
        # few tokens of a small model in fp32
        {"name": "gradient, small model", "op": "gradient", "dtype": "f32", "p": 2, "rows": 777, "hidden": 1536,
         "experts": 16, "k": 2, "weighted": True},
        # a training step of eight ranks
        {"name": "gradient, training step", "op": "gradient", "dtype": "bf16", "p": 8, "rows": 2048, "hidden": 7168,
         "experts": 256, "k": 8, "weighted": True},
        # a small model's many small tensors
        {"name": "clip, many small tensors", "op": "clip", "dtype": "f32", "tensors": 400, "elements": 3000000},
        # a rank's shard of a large model's gradients
        {"name": "clip, large tensors", "op": "clip", "dtype": "bf16", "tensors": 300, "elements": 600000000},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "sort", "dispatch", "combine", "gradient", "clip"])
    case = {"op": op}
    if op == "clip":
        case.update(dtype=rng.choice(["f32", "f16", "bf16"]), tensors=log(1, 600), elements=log(1000, 250000000))
        return case
    case["p"] = rng.choice([1, 2, 3, 4, 8])
    if op == "sort":
        case.update(experts=log(4, 512), k=rng.randint(1, 8), padding=rng.random() < 0.5)
        case["rows"] = log(1, (1 << 20) // (case["p"] * case["k"]))
        return case
    case["dtype"] = rng.choice(["f32", "f16", "bf16"])
    # widths of models are multiples of a vector; others have to work
    case["hidden"] = log(300, 9000) if rng.random() < 0.25 else 8 * log(64, 1024)
    if op == "norm":
        case.update(rows=log(1, (1 << 27) // (case["p"] * case["hidden"])), group=rng.choice([0, 32, 64, 128]))
        return case
    case.update(experts=log(4, 256), k=rng.randint(1, 8), weighted=op != "dispatch" or rng.random() < 0.3)
    case["rows"] = log(1, (1 << 28) // (case["p"] * case["hidden"] * case["k"]))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

class State:
    """A case's inputs and outputs and, for the framework's calls, its communicator."""

    def __init__(self, case):
        self.case = case
        self.comm = None

    def communicate(self, ins, outs=None):
        import reducescatter_reduction_gb300 as ccl
        self.ccl = ccl
        self.comm = ccl.ccl_comm_create(len(ins), [t.data_ptr() for t in ins])
        if outs is not None:
            ccl.ccl_comm_set_outputs(self.comm, [t.data_ptr() for t in outs])

    def __del__(self):
        if self.comm is not None:
            self.ccl.ccl_comm_destroy(self.comm)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = State(case)
    if case["op"] == "norm":
        prepare_norm(s, case, g)
    elif case["op"] == "clip":
        prepare_clip(s, case, g)
    else:
        prepare_choices(s, case, g)
        if case["op"] != "sort":
            prepare_rows(s, case, g)
    if own:
        plan(s)
    return s


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def prepare_norm(s, case, g):
    p, rows, hidden = case["p"], case["rows"], case["hidden"]
    dtype = DTYPES[case["dtype"]]
    s.x = [randn(g, rows, hidden).mul_(p ** -0.5).to(dtype) for _ in range(p)]     # partial sums of a layer's rows
    s.residual = randn(g, rows, hidden).mul_(3).to(dtype)
    # a few channels stand out, as they do in trained models
    s.gamma = (1 + 0.2 * randn(g, hidden) + 4 * (randn(g, hidden) > 2.5)).to(dtype)
    s.eps = 1e-6
    s.residual_out = torch.empty_like(s.residual)
    s.width = case["group"] or hidden
    s.groups = -(-hidden // s.width)
    s.q = [torch.empty(rows, hidden, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(p)]
    s.scales = [torch.empty(rows, s.groups, device="cuda") for _ in range(p)]


def capacity_of(case):
    """Rows that a rank's expert buffer has: a quarter more than its share, and some for small batches."""
    return case["rows"] * case["k"] * 5 // 4 + 32


def prepare_choices(s, case, g):
    p, rows, experts = case["p"], case["rows"], case["experts"]
    k = s.k = min(case["k"], experts)
    s.capacity = capacity_of(case)
    lean = randn(g, experts) * 0.5                                                 # some experts are liked more
    s.ids = [(randn(g, rows, experts) + lean).topk(k, dim=1).indices.to(torch.int32) for _ in range(p)]
    s.valid = None
    if case.get("padding"):
        s.valid = [(torch.arange(rows, device="cuda") < max(1, rows - (7 * r * rows) // (100 * p))).to(torch.uint8)
                   for r in range(p)]
    s.slots = [torch.empty(rows, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    s.offsets = torch.empty(experts + p, dtype=torch.int32, device="cuda")


def prepare_rows(s, case, g):
    p, rows, hidden, k = case["p"], case["rows"], case["hidden"], s.k
    dtype = DTYPES[case["dtype"]]
    s.slots = plain_sort(s)["slots"]
    s.weights = None
    if case["weighted"]:
        s.weights = [torch.softmax(randn(g, rows, k), 1) for _ in range(p)]

    # one allocation for all ranks' tokens, one for all ranks' expert rows and a row that belongs to nobody
    s.all_tokens = torch.empty(p * rows, hidden, dtype=dtype, device="cuda")
    s.all_rows = torch.zeros(p * s.capacity + 1, hidden, dtype=dtype, device="cuda")
    s.tokens = list(s.all_tokens.split(rows))
    s.rows = list(s.all_rows[:-1].split(s.capacity))
    if case["op"] in ("dispatch", "gradient"):
        s.all_tokens.copy_(randn(g, p * rows, hidden))
    if case["op"] == "combine":
        s.all_rows.copy_(randn(g, p * s.capacity + 1, hidden))
    if case["op"] == "gradient":
        s.all_experts = randn(g, p * s.capacity + 1, hidden).to(dtype)
        s.experts = list(s.all_experts[:-1].split(s.capacity))
        s.dweights = [torch.empty(rows, k, device="cuda") for _ in range(p)]


def tensor_sizes(case):
    """Sizes of a model's gradient tensors, by kind: matrices, norm vectors, and a tenth of the vectors that are
    copies of another rank's."""
    count, total = case["tensors"], case["elements"]
    r = random.Random(count * 1000003 + total)
    vectors = count // 2
    share = [math.exp(r.gauss(0, 1)) for _ in range(count - vectors)]
    small = [max(1, min(8192, total // (50 * count))) - r.randint(0, 1) for _ in range(vectors)]
    small = [max(1, n) for n in small]
    left = max(len(share), total - sum(small))
    large = [max(1, int(left * w / sum(share))) for w in share]
    copies = vectors // 10
    return large, small[copies:], small[:copies]


def prepare_clip(s, case, g):
    dtype = DTYPES[case["dtype"]]
    kinds = (dtype, torch.float32, dtype)
    s.sizes = tensor_sizes(case)
    # flat buffers, as a data-parallel optimizer keeps them; the tensors are pieces of them
    s.flat = [torch.empty(sum(n), dtype=t, device="cuda") for n, t in zip(s.sizes, kinds)]
    for f in s.flat:
        f.normal_(0, 0.02, generator=g)
    s.clipped = [torch.empty_like(f) for f in s.flat]
    s.norm = torch.zeros(2, device="cuda")
    s.max_norm = 1.0


def plan(s):
    """What a user's program sets up once for these buffers."""
    op = s.case["op"]
    if op == "norm":
        s.communicate(s.x, s.q)
        s.scale_ptrs = [t.data_ptr() for t in s.scales]
    elif op == "sort":
        s.communicate(s.ids)
    elif op == "dispatch" or op == "gradient":
        s.communicate(s.tokens, s.rows)
    elif op == "combine":
        s.communicate(s.rows, s.tokens)
    else:
        s.communicate([s.norm])
        names = {torch.float32: s.ccl.CCL_F32, torch.float16: s.ccl.CCL_F16, torch.bfloat16: s.ccl.CCL_BF16}
        records = []
        for kind, (sizes, f, out) in enumerate(zip(s.sizes, s.flat, s.clipped)):
            at = 0
            for n in sizes:
                records.append(s.ccl.Tensor(f.data_ptr() + at * f.element_size(), out.data_ptr() + at * f.element_size(),
                                            n, names[f.dtype], kind == 2))
                at += n
        s.tensors = (s.ccl.Tensor * len(records))(*records)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return run_own(s)
    return {"norm": plain_norm, "sort": plain_sort, "dispatch": plain_dispatch, "combine": plain_combine,
            "gradient": plain_gradient, "clip": plain_clip}[s.case["op"]](s)


def pointers(tensors):
    return None if tensors is None else [t.data_ptr() for t in tensors]


def run_own(s):
    case, ccl = s.case, s.ccl
    op = case["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "norm":
        ccl.ccl_allreduce_residual_rmsnorm_e4m3(
            s.comm, case["dtype"], case["rows"], case["hidden"], s.residual.data_ptr(), s.residual_out.data_ptr(),
            s.gamma.data_ptr(), s.scale_ptrs, case["group"], s.eps, "allpairs", stream)
        return {"q": s.q, "scales": s.scales, "residual": s.residual_out}
    if op == "sort":
        ccl.ccl_expert_sort(s.comm, case["rows"], case["experts"], s.k, pointers(s.ids), pointers(s.valid), s.capacity,
                            pointers(s.slots), s.offsets.data_ptr(), stream)
        return {"slots": s.slots, "offsets": s.offsets}
    if op == "dispatch":
        ccl.ccl_expert_dispatch(s.comm, case["dtype"], case["rows"], case["hidden"], s.k, pointers(s.slots),
                                pointers(s.weights), s.capacity, stream)
        return {"rows": s.rows}
    if op == "combine":
        ccl.ccl_expert_combine(s.comm, case["dtype"], case["rows"], case["hidden"], s.k, pointers(s.slots),
                               pointers(s.weights), s.capacity, stream)
        return {"tokens": s.tokens}
    if op == "gradient":
        ccl.ccl_expert_combine_grad(s.comm, case["dtype"], case["rows"], case["hidden"], s.k, pointers(s.slots),
                                    pointers(s.weights), pointers(s.experts), s.capacity, pointers(s.dweights), stream)
        return {"rows": s.rows, "weights": s.dweights}
    ccl.ccl_grad_norm(s.comm, s.tensors, s.norm.data_ptr(), stream)
    ccl.ccl_grad_clip(s.comm, s.tensors, s.max_norm, s.norm.data_ptr(), stream)
    return {"norm": s.norm, "clipped": s.clipped}


def plain_norm(s):
    p, rows, hidden = s.case["p"], s.case["rows"], s.case["hidden"]
    dtype = s.residual.dtype
    y = sum(t.float() for t in s.x).to(dtype).float()
    torch.add(y, s.residual.float(), out=y)
    h = y.to(dtype)
    y = h.float()
    inv = torch.rsqrt(y.square().mean(1, keepdim=True) + s.eps)
    y = (y * s.gamma.float()) * inv
    pad = s.groups * s.width - hidden
    y = torch.nn.functional.pad(y, (0, pad)).view(rows, s.groups, s.width)
    scale = (y.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    q = (y / scale[:, :, None]).to(torch.float8_e4m3fn).view(rows, -1)[:, :hidden].contiguous()
    # every rank has a copy
    return {"q": [q.clone() for _ in range(p)], "scales": [scale.clone() for _ in range(p)], "residual": h}


def plain_sort(s):
    case = s.case
    p, rows, experts, k = case["p"], case["rows"], case["experts"], s.k
    e = torch.stack(s.ids).view(-1).long()
    if s.valid is not None:
        e = torch.where(torch.stack(s.valid).view(-1, 1).expand(-1, k).reshape(-1) > 0, e, experts)
    # the experts' ranks: balanced chunks, the larger ones first
    big, small = experts % p, experts // p
    index = torch.arange(experts + 1, device="cuda")
    edge = big * (small + 1)
    owner = torch.where(index < edge, index // (small + 1), big + (index - edge) // max(small, 1)).clamp(max=p - 1)
    first = torch.arange(p + 1, device="cuda")
    first = first * small + first.clamp(max=big)                          # a rank's first expert
    counts = torch.zeros(experts + 1, dtype=torch.int64, device="cuda").scatter_add_(0, e, torch.ones_like(e))
    start = counts.cumsum(0) - counts
    base = start[first]                                                  # entries before a rank's
    order = torch.sort(e, stable=True).indices
    sorted_e = e[order]
    at = torch.arange(e.numel(), device="cuda") - base[owner[sorted_e]]
    slot = torch.where((sorted_e < experts) & (at < s.capacity), owner[sorted_e] * s.capacity + at, -1)
    slots = torch.empty_like(e).scatter_(0, order, slot).to(torch.int32)
    # per rank: its experts' begins, and their end
    place = torch.arange(experts + p, device="cuda")
    rank = torch.searchsorted(first[1:] + torch.arange(1, p + 1, device="cuda"), place, right=True)
    offsets = (start[place - rank] - base[rank]).clamp(max=s.capacity).to(torch.int32)
    return {"slots": list(slots.view(p, rows, k)), "offsets": offsets}


def plain_dispatch(s):
    case = s.case
    slots = torch.stack(s.slots).view(-1, s.k).long()
    slots = torch.where(slots >= 0, slots, s.all_rows.shape[0] - 1)
    if s.weights is None:
        source = s.all_tokens[:, None, :].expand(-1, s.k, -1)
    else:
        w = torch.stack(s.weights).view(-1, s.k)
        source = (s.all_tokens.float()[:, None, :] * w[:, :, None]).to(s.all_rows.dtype)
    s.all_rows[slots.view(-1)] = source.reshape(-1, case["hidden"])
    return {"rows": s.rows}


def plain_combine(s):
    slots = torch.stack(s.slots).view(-1, s.k).long()
    w = torch.stack(s.weights).view(-1, s.k)
    kept = slots >= 0
    at = slots.clamp(min=0)
    y = sum(torch.where(kept[:, j, None], s.all_rows[at[:, j]].float() * w[:, j, None], 0.0) for j in range(s.k))
    return {"tokens": list(y.to(s.all_rows.dtype).split(s.case["rows"]))}


def plain_gradient(s):
    plain_dispatch(s)
    slots = torch.stack(s.slots).view(-1, s.k).long()
    at = slots.clamp(min=0)
    dy = s.all_tokens.float()
    dw = torch.stack([(dy * s.all_experts[at[:, j]].float()).sum(1) for j in range(s.k)], 1)
    dw = torch.where(slots >= 0, dw, 0.0)
    return {"rows": s.rows, "weights": list(dw.view(s.case["p"], -1, s.k))}


def plain_clip(s):
    norm = sum(f.float().square().sum(dtype=torch.float64) for f in s.flat[:2]).sqrt().float()
    factor = (s.max_norm / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": torch.stack([norm, factor]), "clipped": [(f.float() * factor).to(f.dtype) for f in s.flat]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "clip":
        b = BYTES[case["dtype"]]
        large, small, copies = tensor_sizes(case)
        n = sum(large) + sum(small) + sum(copies)
        return {"bytes": 2 * (b * (sum(large) + sum(copies)) + 4 * sum(small)), "flops": 3 * n}
    p, rows = case["p"], case["rows"]
    if case["op"] == "norm":
        b, n = BYTES[case["dtype"]], rows * case["hidden"]
        groups = -(-case["hidden"] // (case["group"] or case["hidden"]))
        return {"bytes": n * (p * (b + 1) + 2 * b) + p * rows * groups * 4 + case["hidden"] * b, "flops": n * (p + 7)}
    k = min(case["k"], case["experts"])
    tokens = p * rows
    if case["op"] == "sort":
        return {"bytes": tokens * (8 * k + (1 if case["padding"] else 0)) + 4 * (case["experts"] + p),
                "flops": 2 * tokens * k}
    b, n = BYTES[case["dtype"]], tokens * case["hidden"]
    lists = tokens * k * (8 if case["weighted"] else 4)
    if case["op"] == "gradient":
        return {"bytes": n * b * (1 + 2 * k) + lists + 4 * tokens * k, "flops": 3 * n * k}
    return {"bytes": n * b * (1 + k) + lists, "flops": n * k * (2 if case["weighted"] else 0)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "sort":
        return None                                                      # whole numbers
    s = prepare(case, seed)
    return {"norm": exact_norm, "dispatch": exact_dispatch, "combine": exact_combine, "gradient": exact_gradient,
            "clip": exact_clip}[case["op"]](s, case)


def exact_norm(s, case):
    """Row by row of the definition; the sum and the merged residual are of the element type."""
    y = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device="cuda")
    for x in s.x:
        y += x.double()
    h = (y.to(s.residual.dtype).double() + s.residual.double()).to(s.residual.dtype)
    out = h.double() * s.gamma.double() / (h.double().pow(2).sum(1, keepdim=True) / case["hidden"] + s.eps).sqrt()
    scale = torch.empty(case["rows"], s.groups, dtype=torch.float64, device="cuda")
    for i in range(s.groups):
        part = out[:, i * s.width:(i + 1) * s.width]
        scale[:, i] = (part.abs().max(1).values / 448).clamp(min=2.0 ** -126)
        part /= scale[:, i:i + 1]
    p = case["p"]
    return {"q": [out] * p, "scales": [scale] * p, "residual": h.double()}


def pairs(s):
    """(token, choice, row) of the choices that have a row."""
    slots = torch.cat([t.view(-1) for t in s.slots]).long()
    entry = torch.nonzero(slots >= 0).view(-1)
    return entry // s.k, entry % s.k, slots[entry]


def exact_dispatch(s, case):
    token, choice, row = pairs(s)
    out = torch.zeros(case["p"] * s.capacity, case["hidden"], dtype=torch.float64, device="cuda")
    w = torch.cat(s.weights).double() if s.weights else None
    for j in range(s.k):
        of = choice == j
        source = s.all_tokens[token[of]].double()
        if w is not None:
            source *= w[token[of], j][:, None]
        out.index_copy_(0, row[of], source)
    return {"rows": list(out.split(s.capacity))}


def exact_combine(s, case):
    token, choice, row = pairs(s)
    w = torch.cat(s.weights).double()
    out = torch.zeros(case["p"] * case["rows"], case["hidden"], dtype=torch.float64, device="cuda")
    for j in range(s.k):
        of = choice == j
        out.index_add_(0, token[of], s.all_rows[row[of]].double() * w[token[of], j][:, None])
    return {"tokens": list(out.split(case["rows"]))}


def exact_gradient(s, case):
    token, choice, row = pairs(s)
    dw = torch.zeros(case["p"] * case["rows"], s.k, dtype=torch.float64, device="cuda")
    for j in range(s.k):
        of = choice == j
        dw[token[of], j] = torch.einsum("ij,ij->i", s.all_tokens[token[of]].double(), s.all_experts[row[of]].double())
    return {**exact_dispatch(s, case), "weights": list(dw.split(case["rows"]))}


def exact_clip(s, case):
    total = sum(float(part.double().pow(2).sum()) for f in s.flat[:2] for part in f.split(1 << 26))
    norm = math.sqrt(total)
    factor = min(1.0, s.max_norm / (norm + 1e-6))
    return {"norm": torch.tensor([norm, factor], dtype=torch.float64, device="cuda"),
            "clipped": [f.double() * factor for f in s.flat]}

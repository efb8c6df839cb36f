"""The logit operators over rank buffers, as cases to measure: each in a plain
form (elementary torch operations in fp32) and as the calls a user makes.

  rules    penalties for repeated tokens, biases and grammar masks on the
           logits of one decode step, the vocabulary split over p ranks
  distill  the loss against a teacher's top K logits and its gradient, the
           student's vocabulary split over p ranks
  balance  the load-balance loss of a router over p data-parallel ranks, the
           per-expert counts and the gradient of the router's logits
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one request's decode step on one rank: latency
        {"name": "rules, one row", "op": "rules", "dtype": "f32", "p": 1, "rows": 1, "vocab": 32000, "history": 2048,
         "bias": 16, "mask": True},
        # a mid-size batch, a vocabulary that no rank count or vector width divides
        {"name": "rules, odd vocabulary", "op": "rules", "dtype": "f16", "p": 4, "rows": 48, "vocab": 50021,
         "history": 4000, "bias": 300, "mask": True},
        # a full serving batch with long histories, tensor-parallel over eight ranks
        {"name": "rules, full batch", "op": "rules", "dtype": "bf16", "p": 8, "rows": 512, "vocab": 131072,
         "history": 8192, "bias": 64, "mask": True},
        # a few tokens of a small student: latency of loss and gradient at once
        {"name": "distill, few rows", "op": "distill", "dtype": "f32", "p": 1, "rows": 8, "vocab": 32000, "k": 20,
         "steps": "both"},
        # an odd vocabulary over three ranks, ragged teacher lists
        {"name": "distill, odd vocabulary", "op": "distill", "dtype": "bf16", "p": 3, "rows": 700, "vocab": 100003,
         "k": 50, "steps": "both"},
        # one micro-batch of a large-vocabulary student over eight ranks
        {"name": "distill, micro-batch", "op": "distill", "dtype": "bf16", "p": 8, "rows": 4096, "vocab": 131072,
         "k": 64, "steps": "both"},
        # evaluation: the loss alone
        {"name": "distill, loss alone", "op": "distill", "dtype": "f16", "p": 2, "rows": 2048, "vocab": 65536, "k": 128,
         "steps": "forward"},
        # autograd's second half: the gradient from saved statistics
        {"name": "distill, gradient alone", "op": "distill", "dtype": "f32", "p": 2, "rows": 2048, "vocab": 65536,
         "k": 128, "steps": "backward"},
        # a small step of eight ranks: latency
        {"name": "balance, few rows", "op": "balance", "dtype": "bf16", "p": 8, "rows": 64, "experts": 64, "k": 6,
         "steps": "both", "padding": False},
        # a training step: many small experts, padded sequences
        {"name": "balance, training step", "op": "balance", "dtype": "bf16", "p": 8, "rows": 16384, "experts": 256,
         "k": 8, "steps": "both", "padding": True},
        # odd counts of rows and experts, the gradient alone
        {"name": "balance, gradient alone", "op": "balance", "dtype": "f32", "p": 3, "rows": 30011, "experts": 60,
         "k": 4, "steps": "backward", "padding": True},
        # monitoring: loss and counts alone, long rows
        {"name": "balance, loss alone", "op": "balance", "dtype": "f32", "p": 4, "rows": 65536, "experts": 128, "k": 2,
         "steps": "forward", "padding": False},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rules", "distill", "balance"])
    case = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]), "p": rng.choice([1, 2, 3, 4, 8])}
    if op == "balance":
        case.update(experts=log(8, 512), k=rng.randint(1, 8), steps=rng.choice(["forward", "backward", "both"]),
                    padding=rng.random() < 0.5)
        case["rows"] = log(1, (1 << 27) // (case["p"] * case["experts"]))
    else:
        case["vocab"] = log(8000, 260000)
        if op == "rules":
            case["rows"] = log(1, min(512, (1 << 26) // case["vocab"]))
            case.update(history=log(1, 16384), bias=rng.choice([0, log(1, 1000)]), mask=rng.random() < 0.7)
        else:
            case["rows"] = log(1, min(8192, (1 << 28) // case["vocab"]))
            case.update(k=log(1, 256), steps=rng.choice(["forward", "backward", "both"]))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def widths(n, p):
    """p balanced chunks of n, the larger ones first: the library's shards."""
    return [n // p + (1 if r < n % p else 0) for r in range(p)]


class State:
    """A case's inputs, outputs and, for the framework's calls, its communicator."""

    def __init__(self, case):
        self.case = case
        self.comm = None

    def communicate(self):
        import reducescatter_reduction_gb300 as ccl
        self.ccl = ccl
        self.comm = ccl.ccl_comm_create(self.case["p"], [t.data_ptr() for t in self.x])
        ccl.ccl_comm_set_outputs(self.comm, [t.data_ptr() for t in self.y])

    def __del__(self):
        if self.comm is not None:
            self.ccl.ccl_comm_destroy(self.comm)


def split(full, p):
    return [t.contiguous() for t in full.split(widths(full.shape[1], p), dim=1)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = State(case)
    {"rules": prepare_rules, "distill": prepare_distill, "balance": prepare_balance}[case["op"]](s, case, g)
    s.y = [torch.empty_like(t) for t in s.x]
    if own:
        s.communicate()
        if case["op"] == "rules":
            s.rules = s.ccl.LogitRules(
                repetition=s.repetition.data_ptr(), frequency=s.frequency.data_ptr(), presence=s.presence.data_ptr(),
                history=s.history.data_ptr(), history_ld=case["history"], history_len=s.history_len.data_ptr(),
                prompt_len=s.prompt_len.data_ptr())
            if case["bias"]:
                s.rules.bias_offsets = s.bias_offsets.data_ptr()
                s.rules.bias_tokens = s.bias_tokens.data_ptr()
                s.rules.bias_values = s.bias_values.data_ptr()
                s.rules.bias_count = s.bias_tokens.numel()
            if case["mask"]:
                s.rules.mask = s.mask.data_ptr()
                s.rules.mask_rows, s.rules.mask_ld = s.mask.shape
                s.rules.mask_index = s.mask_index.data_ptr()
    return s


def rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def prepare_rules(s, case, g):
    rows, vocab, p, ld = case["rows"], case["vocab"], case["p"], case["history"]
    z = torch.randn(rows, vocab, device="cuda", generator=g).mul_(3).to(DTYPES[case["dtype"]])
    s.x = split(z, p)
    # token lists as text has them: a few frequent tokens, many rare ones
    s.history = (rand(g, rows, ld).pow_(4) * vocab).to(torch.int32)
    length = (rand(g, rows) * (ld + 1)).to(torch.int32)
    length[-1] = ld
    if rows > 1:
        length[0] = 0
    s.history_len = length
    s.prompt_len = (rand(g, rows) * length).to(torch.int32)
    s.repetition = 1 + 0.5 * rand(g, rows)
    s.frequency = rand(g, rows) - 0.2
    s.presence = rand(g, rows) - 0.2
    if case["bias"]:
        count = (rand(g, rows) * (case["bias"] + 1)).to(torch.int32)
        count[-1] = case["bias"]
        s.bias_offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), count.cumsum(0).to(torch.int32)])
        n = int(s.bias_offsets[-1])
        s.bias_tokens = (rand(g, n) * vocab).to(torch.int32)
        s.bias_values = torch.randn(n, device="cuda", generator=g) * 5
    if case["mask"]:
        # a grammar allows few tokens, a block list forbids few; some rows have neither
        words = (vocab + 31) // 32
        kind = torch.arange(rows, device="cuda") % 3
        allow = torch.where(kind == 0, 0.002, 0.98)
        bits = rand(g, rows, words * 32) < allow[:, None]
        shift = torch.arange(32, device="cuda")
        s.mask = (bits.view(rows, words, 32).long() << shift).sum(2).to(torch.int32)
        s.mask_index = torch.where(kind == 2, -1, torch.arange(rows, device="cuda").flip(0)).to(torch.int32)


def prepare_distill(s, case, g):
    rows, vocab, p, k = case["rows"], case["vocab"], case["p"], case["k"]
    z = torch.randn(rows, vocab, device="cuda", generator=g).mul_(2.5)
    # a teacher that agrees with the student in part: its top k of the student's logits and its own view
    parts = [(c + 2.5 * torch.randn(c.shape, device="cuda", generator=g)).topk(k, dim=1) for c in z.split(512)]
    s.teacher = torch.cat([t.values for t in parts])
    s.ids = torch.cat([t.indices for t in parts]).to(torch.int32)
    # ragged lists: entries past a row's own length hold -1; one row has none
    length = (k - rand(g, rows) * min(k, 8)).long()
    if rows > 2:
        length[rows // 2] = 0
    s.ids = torch.where(torch.arange(k, device="cuda") < length[:, None], s.ids, -1).contiguous()
    s.x = split(z.to(DTYPES[case["dtype"]]), p)
    s.weight = rand(g, rows) + 0.5
    s.temperature = 2.0
    s.loss = torch.empty(rows, device="cuda")
    s.stats = torch.empty(rows, 2, device="cuda")
    if case["steps"] == "backward":
        zs = torch.cat([t.float() for t in s.x], 1)
        s.stats[:, 0] = zs.amax(1)
        s.stats[:, 1] = ((zs - s.stats[:, :1]) / s.temperature).exp().sum(1, dtype=torch.float64).log()


def prepare_balance(s, case, g):
    rows, experts, p, k = case["rows"], case["experts"], case["p"], case["k"]
    lean = torch.randn(experts, device="cuda", generator=g) * 0.5   # some experts are liked more
    s.x = [(torch.randn(rows, experts, device="cuda", generator=g) + lean).to(DTYPES[case["dtype"]]) for _ in range(p)]
    k = case["k"] = min(k, experts)
    s.ids = [t.float().topk(k, dim=1).indices.to(torch.int32) for t in s.x]
    s.valid = None
    if case["padding"]:
        s.valid = [(torch.arange(rows, device="cuda") < max(1, rows - (7 * r * rows) // (100 * p))).to(torch.uint8)
                   for r in range(p)]
    s.coef = 0.01
    s.dloss = torch.full((1,), 65536.0, device="cuda")              # a loss scale, as 16-bit gradients need one
    s.counts = torch.empty(p, experts, dtype=torch.int32, device="cuda")
    s.tokens = torch.empty(p, dtype=torch.int32, device="cuda")
    s.loss = torch.empty(1, device="cuda")
    if case["steps"] == "backward":
        s.counts, s.tokens = count_experts(s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (run_own if own else run_plain)(s)


def run_own(s):
    case, ccl = s.case, s.ccl
    stream = torch.cuda.current_stream().cuda_stream
    if case["op"] == "rules":
        ccl.ccl_logit_rules(s.comm, case["dtype"], case["rows"], case["vocab"], s.rules, stream=stream)
        return {"logits": s.y}
    if case["op"] == "distill":
        ccl.ccl_distill_topk(s.comm, case["dtype"], case["steps"], case["rows"], case["vocab"], case["k"],
                             s.ids.data_ptr(), s.teacher.data_ptr(), "f32", s.temperature, s.weight.data_ptr(),
                             s.loss.data_ptr(), s.stats.data_ptr(), stream=stream)
        out = {"grad": s.y} if case["steps"] != "forward" else {}
        return out if case["steps"] == "backward" else {**out, "loss": s.loss, "stats": s.stats}
    ccl.ccl_balance_loss(s.comm, case["dtype"], case["steps"], case["rows"], case["experts"], case["k"],
                         [t.data_ptr() for t in s.ids], [t.data_ptr() for t in s.valid] if s.valid else None, s.coef,
                         s.dloss.data_ptr(), s.counts.data_ptr(), s.tokens.data_ptr(), s.loss.data_ptr(), stream=stream)
    out = {"grad": s.y} if case["steps"] != "forward" else {}
    return out if case["steps"] == "backward" else {**out, "loss": s.loss, "counts": s.counts, "tokens": s.tokens}


def run_plain(s):
    return {"rules": plain_rules, "distill": plain_distill, "balance": plain_balance}[s.case["op"]](s)


def shards(full, like):
    return list(full.to(like[0].dtype).split([t.shape[1] for t in like], dim=1))


def plain_rules(s):
    case = s.case
    rows, vocab = case["rows"], case["vocab"]
    x = torch.cat([t.float() for t in s.x], 1)
    at = torch.arange(case["history"], device="cuda")
    none = torch.full((), vocab, device="cuda")
    token = s.history.long()
    every = torch.where(at < s.history_len[:, None], token, none)
    made = torch.where(at >= s.prompt_len[:, None], every, none)
    one = torch.ones_like(token, dtype=torch.float32)
    seen = torch.zeros(rows, vocab + 1, device="cuda").scatter_add_(1, every, one)[:, :vocab] > 0
    count = torch.zeros(rows, vocab + 1, device="cuda").scatter_add_(1, made, one)[:, :vocab]
    if case["bias"]:
        n = s.bias_tokens.numel()
        row = torch.searchsorted(s.bias_offsets[1:].contiguous(), torch.arange(n, dtype=torch.int32, device="cuda"),
                                 right=True)
        x.view(-1).index_add_(0, row * vocab + s.bias_tokens, s.bias_values)
    rep = s.repetition[:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s.frequency[:, None] * count - s.presence[:, None] * (count > 0)
    if case["mask"]:
        v = torch.arange(vocab, device="cuda")
        word = s.mask[s.mask_index.clamp(min=0).long()][:, v >> 5]
        allowed = ((word >> (v & 31)) & 1).bool() | (s.mask_index[:, None] < 0)
        x = torch.where(allowed, x, -math.inf)
    return {"logits": shards(x, s.x)}


def plain_distill(s):
    case, T = s.case, s.temperature
    z = torch.cat([t.float() for t in s.x], 1)
    valid = s.ids >= 0
    any_ = valid.any(1, keepdim=True)
    t = torch.where(valid, s.teacher, -math.inf)
    u = torch.where(valid, (t - t.amax(1, keepdim=True)) / T, -math.inf)
    logq = torch.where(valid, u - u.exp().sum(1, keepdim=True).log(), 0.0)
    q = torch.where(valid, logq.exp(), 0.0)
    at = s.ids.clamp(min=0).long()
    if case["steps"] == "backward":
        stats = s.stats
    else:
        m = z.amax(1)
        stats = torch.stack([m, ((z - m[:, None]) / T).exp().sum(1).log()], 1)
    d = (z - stats[:, :1]) / T
    logp = d - stats[:, 1:]
    out = {}
    if case["steps"] != "forward":
        grad = logp.exp().scatter_add_(1, at, -q)
        out["grad"] = shards(torch.where(any_, grad * (s.weight[:, None] * T), 0.0), s.x)
    if case["steps"] != "backward":
        out["loss"] = T * T * (q * (logq - logp.gather(1, at))).sum(1)
        out["stats"] = stats
    return out


def count_experts(s):
    ids = torch.stack(s.ids)
    p, rows, k = ids.shape
    valid = torch.stack(s.valid).int() if s.valid else torch.ones(p, rows, dtype=torch.int32, device="cuda")
    counts = torch.zeros(p, s.case["experts"], dtype=torch.int32, device="cuda")
    counts.scatter_add_(1, ids.view(p, -1).long(), valid[:, :, None].expand(p, rows, k).reshape(p, -1))
    return counts, valid.sum(1, dtype=torch.int32)


def plain_balance(s):
    case = s.case
    experts, k = case["experts"], case["k"]
    counts, tokens = (s.counts, s.tokens) if case["steps"] == "backward" else count_experts(s)
    n = tokens.sum().double()
    scale = case_scale(s, n)
    total = counts.sum(0).double()
    mean = total.mean()
    # the gradient goes by differences between the counts: from their mean, in 64 bits, before fp32
    off = ((total - mean) * scale).float()
    x = torch.stack(s.x).float()
    prob = (x - x.amax(2, keepdim=True)).exp()
    prob = prob / prob.sum(2, keepdim=True)
    if s.valid:
        prob = torch.where(torch.stack(s.valid)[:, :, None] > 0, prob, 0.0)
    lean = (prob * off).sum(2, keepdim=True)
    out = {}
    if case["steps"] != "forward":
        out["grad"] = list((prob * (off - lean) * s.dloss).to(s.x[0].dtype))
    if case["steps"] != "backward":
        out["loss"] = (lean.sum(dtype=torch.float64) + n * mean * scale).float().view(1)
        out["counts"], out["tokens"] = counts, tokens
    return out


def case_scale(s, n):
    return s.coef * s.case["experts"] / (s.case["k"] * n * n)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    b = BYTES[case["dtype"]]
    rows = case["rows"]
    if case["op"] == "rules":
        n = rows * case["vocab"]
        history = rows * (case["history"] + 1) // 2
        bias = rows * (case["bias"] + 1) // 2
        size = 2 * n * b + 4 * history + 8 * bias + (n // 12 if case["mask"] else 0)
        return {"bytes": size, "flops": 2 * n + 4 * history}
    if case["op"] == "distill":
        n = rows * case["vocab"]
        moves = 1 if case["steps"] == "forward" else 2
        return {"bytes": moves * n * b + rows * (8 * case["k"] + 16),
                "flops": n * {"forward": 4, "backward": 5, "both": 7}[case["steps"]]}
    n = case["p"] * rows
    k = min(case["k"], case["experts"])
    moves = 1 if case["steps"] == "forward" else 2
    return {"bytes": n * (case["experts"] * b * moves + (0 if case["steps"] == "backward" else 4 * k)
                          + (1 if case["padding"] else 0)),
            "flops": n * case["experts"] * {"forward": 6, "backward": 8, "both": 8}[case["steps"]]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rules": exact_rules, "distill": exact_distill, "balance": exact_balance}[case["op"]](s, case)


def cut(full, p):
    edges = np.cumsum([0] + widths(full.shape[1], p))
    return [full[:, a:b] for a, b in zip(edges[:-1], edges[1:])]


def exact_rules(s, case):
    """Row by row on the host, from the definition."""
    rows, vocab = case["rows"], case["vocab"]
    y = torch.cat([t.double() for t in s.x], 1).cpu().numpy()
    history, length, prompt = s.history.cpu().numpy(), s.history_len.cpu().numpy(), s.prompt_len.cpu().numpy()
    rep, freq, pres = (t.double().cpu().numpy() for t in (s.repetition, s.frequency, s.presence))
    if case["bias"]:
        offsets, tokens = s.bias_offsets.cpu().numpy(), s.bias_tokens.cpu().numpy()
        values = s.bias_values.double().cpu().numpy()
    if case["mask"]:
        words, index = s.mask.cpu().numpy(), s.mask_index.cpu().numpy()
    for i in range(rows):
        if case["bias"]:
            part = slice(offsets[i], offsets[i + 1])
            np.add.at(y[i], tokens[part], values[part])
        every = np.unique(history[i, :length[i]])
        y[i, every] = np.where(y[i, every] > 0, y[i, every] / rep[i], y[i, every] * rep[i])
        made, times = np.unique(history[i, prompt[i]:length[i]], return_counts=True)
        y[i, made] -= freq[i] * times + pres[i]
        if case["mask"] and index[i] >= 0:
            bits = np.unpackbits(words[index[i]].view(np.uint8), bitorder="little")[:vocab]
            y[i, bits == 0] = -np.inf
    return {"logits": cut(y, case["p"])}


def exact_distill(s, case):
    """A block of rows at a time, in fp64."""
    T, p = s.temperature, case["p"]
    rows = case["rows"]
    grads, losses, stats = [[] for _ in range(p)], [], []
    for a in range(0, rows, 256):
        z = torch.cat([t[a:a + 256] for t in s.x], 1).double()
        m = z.max(1, keepdim=True).values
        e = torch.exp((z - m) / T)
        total = e.sum(1, keepdim=True)
        ids, t = s.ids[a:a + 256].long(), s.teacher[a:a + 256].double() / T
        has = (ids >= 0)
        w = torch.exp(t - t.max(1, keepdim=True).values) * has
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        if case["steps"] != "forward":
            prob = (e / total) * has.any(1, keepdim=True)
            prob.scatter_add_(1, ids.clamp(min=0), -w)
            prob *= (s.weight[a:a + 256].double() * T)[:, None]
            for r, part in enumerate(prob.to(torch.float32 if z.numel() * (rows // 256 + 1) > 1 << 28 else z.dtype)
                                     .split(widths(case["vocab"], p), dim=1)):
                grads[r].append(part)
        if case["steps"] != "backward":
            at = z.gather(1, ids.clamp(min=0))
            logp = (at - m) / T - total.log()
            losses.append(T * T * (torch.xlogy(w, w) - w * logp).sum(1))
            stats.append(torch.cat([m, total.log()], 1))
    out = {}
    if case["steps"] != "forward":
        out["grad"] = [torch.cat(g) for g in grads]
    if case["steps"] != "backward":
        out["loss"], out["stats"] = torch.cat(losses), torch.cat(stats)
    return out


def exact_balance(s, case):
    """loss = coef E sum_e f_e P_e and its derivative, rank by rank in fp64."""
    experts, k, p = case["experts"], case["k"], case["p"]
    keep = [torch.ones(case["rows"], dtype=torch.bool, device="cuda") for _ in range(p)]
    if s.valid:
        keep = [v.bool() for v in s.valid]
    n = sum(int(v.sum()) for v in keep)
    hits = sum(torch.bincount(i[v].view(-1).long(), minlength=experts) for i, v in zip(s.ids, keep)).double()
    f = hits / (k * n)
    grads, mass = [], torch.zeros(experts, dtype=torch.float64, device="cuda")
    for x, v in zip(s.x, keep):
        e = torch.exp(x.double() - x.double().max(1, keepdim=True).values)
        e = (e / e.sum(1, keepdim=True)) * v[:, None]
        mass += e.sum(0)
        if case["steps"] != "forward":
            grads.append(s.dloss.double() * s.coef * experts / n * e * (f - (e @ f)[:, None]))
    out = {"grad": grads} if case["steps"] != "forward" else {}
    if case["steps"] != "backward":
        out["loss"] = (s.coef * experts * (f * mass).sum() / n).view(1)
        out["counts"] = out["tokens"] = None
    return out

"""The operators on logits where a model uses them: a head whose vocabulary
is split over p ranks, decoding and then learning from a teacher.

  decode    partial sums of the last layer -> AllReduce + residual + RMSNorm
            -> each rank's columns of the head -> penalties, biases and the
            grammar mask -> the most likely token, appended to the history; one
            step is captured in a CUDA graph and replayed
  training  each rank's columns of the head -> loss against the teacher's top
            logits and its gradient, in place -> each rank's part of dx ->
            AllReduce; and the router of p data-parallel ranks -> load-balance
            loss and its gradient

Weights and tokens are random.  For a summary, from the top of the repository:

  PYTHONPATH=. python examples/sharded_head_step.py
"""
import torch

import reducescatter_reduction_gb300 as ccl


def stream():
    return torch.cuda.current_stream().cuda_stream


def shard_widths(n, p):
    """Columns of each rank: balanced, the larger shards first."""
    return [n // p + (r < n % p) for r in range(p)]


def decode(p=4, rows=3, hidden=256, vocab=1003, steps=8, seed=0):
    """Greedy tokens [rows, steps], and the bool [rows, vocab] that the grammar allows."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    prompt, total = 4, 4 + steps
    history = torch.randint(vocab, (rows, total), generator=g, device="cuda", dtype=torch.int32)
    length = torch.full((rows,), prompt, device="cuda", dtype=torch.int32)
    prompt_len = length.clone()
    allowed = torch.rand(rows, vocab, generator=g, device="cuda") < 0.1
    words = (vocab + 31) // 32
    bits = torch.zeros(rows, words * 32, device="cuda", dtype=torch.int64)
    bits[:, :vocab] = allowed
    bits = (bits.view(rows, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32)
    repetition = torch.full((rows,), 1.3, device="cuda")
    frequency = torch.full((rows,), 0.5, device="cuda")
    presence = torch.full((rows,), 0.25, device="cuda")
    bias_offsets = torch.arange(rows + 1, device="cuda", dtype=torch.int32)      # one entry a row
    bias_tokens = torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    bias_values = torch.full((rows,), 0.5, device="cuda")
    rules = ccl.LogitRules(
        repetition=repetition.data_ptr(), frequency=frequency.data_ptr(), presence=presence.data_ptr(),
        history=history.data_ptr(), history_ld=total, history_len=length.data_ptr(), prompt_len=prompt_len.data_ptr(),
        bias_offsets=bias_offsets.data_ptr(), bias_tokens=bias_tokens.data_ptr(), bias_values=bias_values.data_ptr(),
        bias_count=rows, mask=mask.data_ptr(), mask_rows=rows, mask_ld=words)

    embedding, gamma, residual = rand(vocab, hidden), rand(hidden), rand(rows, hidden)
    layer = [rand(hidden, hidden) / hidden ** 0.5 for _ in range(p)]             # stands for the ranks' layers
    partial = [torch.empty(rows, hidden, device="cuda", dtype=torch.bfloat16) for _ in range(p)]
    normed = [torch.empty_like(x) for x in partial]
    residual_out = torch.empty_like(residual)
    head = [rand(w, hidden) / hidden ** 0.5 for w in shard_widths(vocab, p)]
    logits = [torch.empty(rows, w, device="cuda", dtype=torch.bfloat16) for w in shard_widths(vocab, p)]
    hidden_comm = ccl.ccl_comm_create(p, [x.data_ptr() for x in partial])
    ccl.ccl_comm_set_outputs(hidden_comm, [x.data_ptr() for x in normed])
    logit_comm = ccl.ccl_comm_create(p, [x.data_ptr() for x in logits])          # outputs = inputs: in place
    now, out = torch.empty(rows, 1, device="cuda", dtype=torch.int64), torch.empty(rows, 1, device="cuda", dtype=torch.int64)

    def step():
        torch.sub(length.view(rows, 1), 1, out=now)
        x = embedding[history.gather(1, now).long().view(-1)]
        for r in range(p):
            torch.matmul(x, layer[r], out=partial[r])
        ccl.ccl_allreduce_residual_rmsnorm(hidden_comm, "bf16", rows, hidden, residual.data_ptr(),
                                           residual_out.data_ptr(), gamma.data_ptr(), 1e-6, "ring", stream())
        for r in range(p):
            torch.matmul(normed[r], head[r].t(), out=logits[r])
        ccl.ccl_logit_rules(logit_comm, "bf16", rows, vocab, rules, 0, stream())
        torch.argmax(torch.cat(logits, 1), 1, keepdim=True, out=out)
        history.scatter_(1, now + 1, out.int())
        length.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                                   # the first token, and the warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps - 1):
        graph.replay()
    for comm in (hidden_comm, logit_comm):
        ccl.ccl_comm_check(comm)
        ccl.ccl_comm_destroy(comm)
    return history[:, prompt:].clone(), allowed


def train(p=4, rows=64, hidden=128, vocab=1003, k=16, experts=32, choices=4, steps=10, temperature=2.0, coef=0.01,
          seed=0):
    """Per step: (mean distillation loss, balance loss)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, hidden, generator=g, device="cuda")
    teacher = x @ torch.randn(vocab, hidden, generator=g, device="cuda").t() / hidden ** 0.5 * 4
    teacher_logits, teacher_ids = teacher.topk(k, 1)
    teacher_ids, teacher_logits = teacher_ids.int(), teacher_logits.contiguous()
    weight = torch.full((rows,), 1.0 / rows, device="cuda")                      # the mean over the rows
    head = [torch.randn(w, hidden, generator=g, device="cuda") / hidden ** 0.5 for w in shard_widths(vocab, p)]
    logits = [torch.empty(rows, h.shape[0], device="cuda") for h in head]
    dx = [torch.empty(rows, hidden, device="cuda") for _ in range(p)]
    loss = torch.empty(rows, device="cuda")
    head_comm = ccl.ccl_comm_create(p, [t.data_ptr() for t in logits])
    dx_comm = ccl.ccl_comm_create(p, [t.data_ptr() for t in dx])

    # the router: p data-parallel ranks, each with `rows` tokens of its own
    tokens = [torch.randn(rows, hidden, generator=g, device="cuda") for _ in range(p)]
    router = torch.randn(experts, hidden, generator=g, device="cuda") / hidden ** 0.5
    router[:choices] += 0.05                                                     # not balanced to begin with
    for t in tokens:
        t += 0.5
    valid = [torch.ones(rows, device="cuda", dtype=torch.uint8) for _ in range(p)]
    valid[-1][rows // 2:] = 0                                                    # padding
    routes = [torch.empty(rows, experts, device="cuda") for _ in range(p)]
    counts = torch.empty(p, experts, device="cuda", dtype=torch.int32)
    valid_rows = torch.empty(p, device="cuda", dtype=torch.int32)
    balance = torch.empty(1, device="cuda")
    route_comm = ccl.ccl_comm_create(p, [t.data_ptr() for t in routes])

    seen = []
    for _ in range(steps):
        for r in range(p):
            torch.matmul(x, head[r].t(), out=logits[r])
        ccl.ccl_distill_topk(head_comm, "f32", "both", rows, vocab, k, teacher_ids.data_ptr(),
                             teacher_logits.data_ptr(), "f32", temperature, row_weight=weight.data_ptr(),
                             loss=loss.data_ptr(), stream=stream())              # logits: their gradient
        for r in range(p):
            torch.matmul(logits[r], head[r], out=dx[r])
        ccl.ccl_allreduce(dx_comm, "sum", "f32", rows * hidden, "ring", stream())
        for r in range(p):
            torch.matmul(tokens[r], router.t(), out=routes[r])
        ids = [t.topk(choices, 1).indices.int() for t in routes]
        ccl.ccl_balance_loss(route_comm, "f32", "both", rows, experts, choices, [t.data_ptr() for t in ids],
                             [t.data_ptr() for t in valid], coef, dloss=0, counts=counts.data_ptr(),
                             tokens=valid_rows.data_ptr(), loss=balance.data_ptr(), stream=stream())
        seen.append((loss.mean().item(), balance.item()))
        for r in range(p):
            head[r] -= 0.5 * (logits[r].t() @ x)
            router -= 20.0 * (routes[r].t() @ tokens[r])
        x -= 0.5 * dx[0]
    for comm in (head_comm, dx_comm, route_comm):
        ccl.ccl_comm_check(comm)
        ccl.ccl_comm_destroy(comm)
    return seen


if __name__ == "__main__":
    tokens, allowed = decode()
    print("decoded", tokens.tolist(), "all allowed:", bool(allowed.gather(1, tokens.long()).all()))
    for i, (distill, balance) in enumerate(train()):
        print(f"step {i}: distillation {distill:.4f}  balance {balance:.5f}")

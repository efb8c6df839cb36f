"""The operators around layers where a model uses them: a layer whose experts
are split over p ranks, decoding and then learning.

  decode    partial sums of the layer before -> AllReduce + residual + RMSNorm
            with an 8-bit output -> router -> the choices' rows -> codes and
            scales to their experts -> the experts' products -> back to the
            tokens, weighted; one step is captured in a CUDA graph and replayed
  training  the same layer in fp32 over the tokens of p data-parallel ranks:
            sort, dispatch, experts, combine; combine's gradient, the experts',
            dispatch's gradient (a combine without weights), the router's with
            its balance loss -> AllReduce of the router's gradients, which all
            ranks have -> global norm, a copy counted once, and clipping

Weights and tokens are random.  For a summary, from the top of the repository:

  PYTHONPATH=. python examples/expert_layer_step.py
"""
import torch

import reducescatter_reduction_gb300 as ccl


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptrs(tensors):
    return [t.data_ptr() for t in tensors]


def expert_counts(n, p):
    """Experts of each rank: balanced, the larger parts first."""
    return [n // p + (r < n % p) for r in range(p)]


class Comms:
    """Communicators over pairs of (inputs, outputs), checked and destroyed at the end."""

    def __init__(self):
        self.all = []

    def over(self, ins, outs=None):
        comm = ccl.ccl_comm_create(len(ins), ptrs(ins))
        if outs is not None:
            ccl.ccl_comm_set_outputs(comm, ptrs(outs))
        self.all.append(comm)
        return comm

    def close(self):
        for comm in self.all:
            ccl.ccl_comm_check(comm)
            ccl.ccl_comm_destroy(comm)


def experts_of_rows(offsets, r, counts, capacity):
    """(expert of each row of rank r's buffer, counted from its first; whether the row is taken)."""
    first = sum(counts[:r])
    part = offsets[first + r:first + r + counts[r] + 1]
    row = torch.arange(capacity, device="cuda", dtype=torch.int32)
    of = torch.searchsorted(part[1:].contiguous(), row, right=True)
    return of.clamp(max=max(0, counts[r] - 1)), row < part[-1]


def decode(p=4, rows=6, hidden=256, experts=10, k=3, group=32, steps=3, seed=0):
    """Per step, (inputs, outputs) of the layer: what a plain computation needs to check it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    bf16 = lambda t: t.bfloat16()
    counts, capacity, groups = expert_counts(experts, p), rows * k * p, hidden // group
    partial = [torch.empty(rows, hidden, device="cuda", dtype=torch.bfloat16) for _ in range(p)]
    residual, gamma = bf16(rand(rows, hidden)), bf16(1 + 0.1 * rand(hidden))
    codes = [torch.empty(rows, hidden, device="cuda", dtype=torch.uint8) for _ in range(p)]
    scales = [torch.empty(rows, groups, device="cuda") for _ in range(p)]
    router = rand(experts, hidden) / hidden ** 0.5
    weight = [rand(n, hidden, hidden) / hidden ** 0.5 for n in counts]
    # after the AllReduce every rank has all rows: rank r sends rows r, r + p, ... and the others are padding
    mine = [(torch.arange(rows, device="cuda") % p == r).to(torch.uint8) for r in range(p)]
    ids = [torch.empty(rows, k, device="cuda", dtype=torch.int32) for _ in range(p)]
    share = [torch.empty(rows, k, device="cuda") for _ in range(p)]
    slots = [torch.empty(rows, k, device="cuda", dtype=torch.int32) for _ in range(p)]
    offsets = torch.empty(experts + p, device="cuda", dtype=torch.int32)
    expert_codes = [torch.zeros(capacity, hidden, device="cuda", dtype=torch.uint8) for _ in range(p)]
    expert_scales = [torch.zeros(capacity, groups, device="cuda") for _ in range(p)]
    expert_rows = [torch.zeros(capacity, hidden, device="cuda", dtype=torch.bfloat16) for _ in range(p)]
    out = [torch.empty(rows, hidden, device="cuda", dtype=torch.bfloat16) for _ in range(p)]
    comms = Comms()
    norm_comm, code_comm = comms.over(partial, codes), comms.over(codes, expert_codes)
    scale_comm, back_comm = comms.over(scales, expert_scales), comms.over(expert_rows, out)

    def dequantised(q, s):
        return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(group, 1)

    def step():
        ccl.ccl_allreduce_residual_rmsnorm_e4m3(norm_comm, "bf16", rows, hidden, residual.data_ptr(), residual.data_ptr(),
                                                gamma.data_ptr(), ptrs(scales), group, 1e-6, "ring", stream())
        for r in range(p):
            top = (dequantised(codes[r], scales[r]) @ router.t()).topk(k, 1)
            ids[r].copy_(top.indices)
            share[r].copy_(torch.softmax(top.values, 1))
        ccl.ccl_expert_sort(code_comm, rows, experts, k, ptrs(ids), ptrs(mine), capacity, ptrs(slots), offsets.data_ptr(),
                            stream())
        ccl.ccl_expert_dispatch(code_comm, "i32", rows, hidden // 4, k, ptrs(slots), None, capacity, stream())
        ccl.ccl_expert_dispatch(scale_comm, "f32", rows, groups, k, ptrs(slots), None, capacity, stream())
        for r in range(p):
            if counts[r]:
                of, taken = experts_of_rows(offsets, r, counts, capacity)
                y = torch.bmm(dequantised(expert_codes[r], expert_scales[r])[:, None], weight[r][of])[:, 0]
                expert_rows[r].copy_(torch.where(taken[:, None], y, 0.0))
        ccl.ccl_expert_combine(back_comm, "bf16", rows, hidden, k, ptrs(slots), ptrs(share), capacity, stream())

    def load():
        for t in partial:
            t.copy_(rand(rows, hidden) / p ** 0.5)
        return [t.clone() for t in partial], residual.clone()

    seen = []
    graph = None
    for i in range(steps):
        inputs = load()
        if graph is not None:
            graph.replay()
        else:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()                                              # the first step, and the warm-up
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        seen.append({"partial": inputs[0], "residual": inputs[1], "residual_out": residual.clone(),
                     "x": dequantised(codes[0], scales[0]), "out": sum(t.float() for t in out)})
    comms.close()
    return seen, {"gamma": gamma, "router": router, "weight": torch.cat(weight), "k": k}


class Layer:
    """y = x + sum_j share_j tanh(x A_(expert j)), the experts' matrices A split over the ranks, and its training step."""

    def __init__(self, p=4, rows=40, hidden=48, experts=7, k=2, coef=0.02, max_norm=0.5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        empty = lambda *s, dtype=torch.float32: torch.zeros(*s, device="cuda", dtype=dtype)
        self.p, self.rows, self.hidden, self.experts, self.k = p, rows, hidden, experts, k
        self.coef, self.max_norm = coef, max_norm
        self.counts, self.capacity = expert_counts(experts, p), rows * k * p
        c, C = self.counts, self.capacity
        self.x = [rand(rows, hidden) for _ in range(p)]
        self.target = [rand(rows, hidden) for _ in range(p)]
        self.valid = [torch.ones(rows, device="cuda", dtype=torch.uint8) for _ in range(p)]
        self.valid[-1][rows // 2:] = 0                                  # padding
        self.router = rand(experts, hidden) / hidden ** 0.5
        self.weight = [rand(n, hidden, hidden) / hidden ** 0.5 for n in c]
        tokens, rows_of = (lambda: [empty(rows, hidden) for _ in range(p)]), (lambda: [empty(C, hidden) for _ in range(p)])
        self.logits, self.ids = [empty(rows, experts) for _ in range(p)], [empty(rows, k, dtype=torch.int32) for _ in range(p)]
        self.dlogits = [empty(rows, experts) for _ in range(p)]
        self.share, self.dshare = [empty(rows, k) for _ in range(p)], [empty(rows, k) for _ in range(p)]
        self.slots = [empty(rows, k, dtype=torch.int32) for _ in range(p)]
        self.offsets = empty(experts + p, dtype=torch.int32)
        self.xe, self.ze, self.dze, self.dxe = rows_of(), rows_of(), rows_of(), rows_of()
        self.sum, self.dy, self.dx = tokens(), tokens(), tokens()
        self.counted, self.tokens, self.balance = empty(p, experts, dtype=torch.int32), empty(p, dtype=torch.int32), empty(1)
        self.drouter, self.dweight = [empty(experts, hidden) for _ in range(p)], [empty(n, hidden, hidden) for n in c]
        self.norm = empty(2)
        self.comms = Comms()
        over = self.comms.over
        self.there, self.back = over(self.x, self.xe), over(self.ze, self.sum)
        self.back_grad, self.there_grad = over(self.dy, self.dze), over(self.dxe, self.dx)
        self.route, self.reduce = over(self.logits, self.dlogits), over(self.drouter)
        grads = [ccl.Tensor(t.data_ptr(), t.data_ptr(), t.numel(), ccl.CCL_F32, 0) for t in self.dweight if t.numel()]
        grads += [ccl.Tensor(t.data_ptr(), t.data_ptr(), t.numel(), ccl.CCL_F32, r) for r, t in enumerate(self.drouter)]
        self.grads = (ccl.Tensor * len(grads))(*grads)

    def gradients(self):
        """One forward and backward pass; the loss (mean square error over the valid rows, and the balance loss)."""
        p, rows, hidden, experts, k, C = self.p, self.rows, self.hidden, self.experts, self.k, self.capacity
        for r in range(p):
            torch.matmul(self.x[r], self.router.t(), out=self.logits[r])
            top = self.logits[r].topk(k, 1)
            self.ids[r].copy_(top.indices)
            self.share[r].copy_(torch.softmax(top.values, 1))
        ccl.ccl_expert_sort(self.there, rows, experts, k, ptrs(self.ids), ptrs(self.valid), C, ptrs(self.slots),
                            self.offsets.data_ptr(), stream())
        ccl.ccl_expert_dispatch(self.there, "f32", rows, hidden, k, ptrs(self.slots), None, C, stream())
        of = [experts_of_rows(self.offsets, r, self.counts, C) for r in range(p)]
        for r in range(p):
            if self.counts[r]:
                z = torch.tanh(torch.bmm(self.xe[r][:, None], self.weight[r][of[r][0]])[:, 0])
                self.ze[r].copy_(torch.where(of[r][1][:, None], z, 0.0))
        ccl.ccl_expert_combine(self.back, "f32", rows, hidden, k, ptrs(self.slots), ptrs(self.share), C, stream())
        valid = [v.float()[:, None] for v in self.valid]
        n = sum(v.sum() for v in valid) * hidden
        loss = 0.0
        for r in range(p):
            off = (self.x[r] + self.sum[r] - self.target[r]) * valid[r]
            loss = loss + off.square().sum() / n
            self.dy[r].copy_(2 * off / n)
        ccl.ccl_expert_combine_grad(self.back_grad, "f32", rows, hidden, k, ptrs(self.slots), ptrs(self.share), ptrs(self.ze),
                                    C, ptrs(self.dshare), stream())
        for r in range(p):
            if self.counts[r]:
                e, taken = of[r]
                dpre = torch.where(taken[:, None], self.dze[r] * (1 - self.ze[r].square()), 0.0)
                self.dxe[r].copy_(torch.bmm(dpre[:, None], self.weight[r][e].transpose(1, 2))[:, 0])
                xe = torch.where(taken[:, None], self.xe[r], 0.0)
                self.dweight[r].zero_().index_add_(0, e, xe[:, :, None] * dpre[:, None, :])
        ccl.ccl_expert_combine(self.there_grad, "f32", rows, hidden, k, ptrs(self.slots), None, C, stream())
        ccl.ccl_balance_loss(self.route, "f32", "both", rows, experts, k, ptrs(self.ids), ptrs(self.valid), self.coef, 0,
                             self.counted.data_ptr(), self.tokens.data_ptr(), self.balance.data_ptr(), stream())
        for r in range(p):
            ds = self.share[r] * (self.dshare[r] - (self.share[r] * self.dshare[r]).sum(1, keepdim=True))
            self.dlogits[r].scatter_add_(1, self.ids[r].long(), ds)
            torch.matmul(self.dlogits[r].t(), self.x[r], out=self.drouter[r])
            self.dx[r] += self.dy[r] + self.dlogits[r] @ self.router
        ccl.ccl_allreduce(self.reduce, "sum", "f32", experts * hidden, "ring", stream())
        return loss + self.balance[0]

    def clip(self):
        """Clips the gradients in place; (global norm, factor) stay on the device."""
        ccl.ccl_grad_norm(self.reduce, self.grads, self.norm.data_ptr(), stream())
        ccl.ccl_grad_clip(self.reduce, self.grads, self.max_norm, self.norm.data_ptr(), stream())

    def step(self, rate=0.5):
        loss = self.gradients()
        self.clip()
        self.router -= rate * self.drouter[0]
        for w, dw in zip(self.weight, self.dweight):
            w -= rate * dw
        return loss

    def close(self):
        self.comms.close()


if __name__ == "__main__":
    seen, _ = decode()
    print("decoded", len(seen), "steps, mean square of the outputs", [round(float(s["out"].square().mean()), 4) for s in seen])
    layer = Layer()
    for i in range(10):
        loss = layer.step()
        print(f"step {i}: loss {float(loss):.4f}  gradient norm {float(layer.norm[0]):.4f}  factor {float(layer.norm[1]):.4f}")
    layer.close()

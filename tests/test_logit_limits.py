"""What the logit operators accept at the ends of their arguments' ranges: the
refusals on the CPU, the results there on a GPU."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import rng
from test_logit_refusals import BAD, OK, distill_call, front, status      # noqa: F401 (front: a fixture)
from test_logit_rules import Rules, check


@pytest.mark.cpu
@pytest.mark.parametrize("temperature,want", [
    (1e-45, BAD), (1e-40, BAD), (4.2e-39, BAD), (4.3e-39, OK), (1e-38, OK), (1e-30, OK), (3e38, OK), (-1e-40, BAD)])
def test_temperatures_whose_reciprocal_is_infinite(front, temperature, want):      # noqa: F811
    assert status(front, distill_call(front, temperature=temperature)) == (want, int(want == OK))
    if want == BAD:
        assert b"temperature" in front.fake_message()


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


@pytest.mark.gpu
@pytest.mark.parametrize("steps", ["forward", "both"])
@pytest.mark.parametrize("T", [1e-38, 1e-30, 1e-22, 1e-10])
def test_losses_at_temperatures_whose_square_underflows(gpu, steps, T):
    """The student has its weight on token 0, the teacher on token 3, d below it: the loss is T^2 (d / T) = T d.  Roundings:
    d / T, two products with T, and T itself (to fp32, which the wanted value has already)."""
    rows, vocab = 4, 1000
    d = np.array([0.25, 1.0, 2.0, 1.5])
    z = np.full((rows, vocab), -5.0, dtype=np.float32)
    z[:, 0], z[:, 3] = 0.0, -d
    logits = [torch.from_numpy(z[:, :500].copy()).cuda(), torch.from_numpy(z[:, 500:].copy()).cuda()]
    ids = torch.tensor([[3, 7]] * rows, dtype=torch.int32, device="cuda")
    teacher = torch.tensor([[2.0, 1.0]] * rows, device="cuda")
    loss = torch.empty(rows, device="cuda")
    comm = ccl.ccl_comm_create(2, [x.data_ptr() for x in logits])
    ccl.ccl_distill_topk(comm, "f32", steps, rows, vocab, 2, ids.data_ptr(), teacher.data_ptr(), temperature=T, loss=loss.data_ptr(),
                         stream=torch.cuda.current_stream().cuda_stream)
    ccl.ccl_comm_check(comm)
    ccl.ccl_comm_destroy(comm)
    want = float(np.float32(T)) * d
    err = np.abs(loss.double().cpu().numpy() - want)
    assert (err <= 8 * 2.0 ** -24 * want + 2.0 ** -149).all(), (loss.tolist(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [1000, 300000])
def test_bias_entries_at_the_end_of_the_longest_list(gpu, vocab):
    """2^31 - 1 entries: the blocks that a row's last entries are read in end beyond 2^31."""
    n, some, rows = 2 ** 31 - 1, 600, 4
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    g = rng(1)
    tokens, values = (torch.empty(n, dtype=t, device="cuda") for t in (torch.int32, torch.float32))
    h = {"bias_offsets": np.array([0, some, some, some, some], dtype=np.int32),
         "bias_tokens": g.integers(0, vocab, some).astype(np.int32), "bias_values": g.normal(0, 2, some).astype(np.float32)}
    tokens[-some:], values[-some:] = torch.from_numpy(h["bias_tokens"]).cuda(), torch.from_numpy(h["bias_values"]).cuda()
    offsets = torch.tensor([n - some, n, n, n, n], dtype=torch.int32, device="cuda")
    rules = Rules(**h)
    rules.s = ccl.LogitRules(bias_offsets=offsets.data_ptr(), bias_tokens=tokens.data_ptr(), bias_values=values.data_ptr(), bias_count=n)
    check(g.normal(0, 4, (rows, vocab)), 2, "f32", rules)

"""What the logit operators accept at the ends of their arguments' ranges: the
refusals on the CPU, the results there on a GPU."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import rng
from test_logit_refusals import BAD, OK, distill_call, front, status      # noqa: F401 (front: a fixture)


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

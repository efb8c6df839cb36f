"""GPU tests of ccl_balance_loss at the ends of its ranges: logits of large
magnitude, no rows."""
import numpy as np
import pytest
import torch

import reducescatter_reduction_gb300 as ccl
from ccl_testutil import ensure_built
from logit_testutil import rng, stream
from test_balance import check, choices

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E", [8, 32, 33, 600, 700, 1500])
@pytest.mark.parametrize("steps", ["both", "forward", "each"])
def test_logits_of_large_magnitude(dtype, E, steps):
    """Rows that are one large value throughout (all experts masked with a finite number) have a uniform softmax, rows
    that are it in part have none there, and rows far from zero are what their differences make of them."""
    g = rng(E)
    values = [v * s for v in (1e5, 1e6, 2e7, 1e9, 3e9, 1e10, 1e20, 1e30, 1e38, 3e38) for s in (1, -1)]
    x = g.normal(0, 2, (4 * len(values), E))
    for i, v in enumerate(values):
        x[4 * i] = v                                        # throughout
        x[4 * i + 1, ::3] = -abs(v)                         # masked in part
        x[4 * i + 2] += v                                   # far from zero: the type keeps what it keeps of it
        x[4 * i + 3] = v * (1 - 0.5 * g.random(E))          # differences as large as the values
    check([x, x[::-1].copy()], choices(len(x), E, 3, 2, 8), dtype, steps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,E", [(2, 16), (3, 17), (1, 2000), (64, 32), (8, 1024), (16, 1024), (8, 3000)])
@pytest.mark.parametrize("padded", [False, True])
def test_no_rows_count_nothing(dtype, p, E, padded):
    """What lies where the lists of no rows begin are expert numbers and valid rows, and nobody's."""
    logits = torch.ones(64, device="cuda")
    ids = torch.arange(64, dtype=torch.int32, device="cuda") % 4
    valid = torch.ones(64, dtype=torch.uint8, device="cuda")
    counts = torch.full((p, E), 5, dtype=torch.int32, device="cuda")
    tokens = torch.full((p,), 5, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), 5.0, device="cuda")
    comm = ccl.ccl_comm_create(p, [logits.data_ptr()] * p)
    for steps in ("forward", "both", "forward"):
        ccl.ccl_balance_loss(comm, dtype, steps, 0, E, 2, [ids.data_ptr()] * p, [valid.data_ptr()] * p if padded else None, 0.1, 0,
                             counts.data_ptr(), tokens.data_ptr(), loss.data_ptr(), stream=stream())
        ccl.ccl_comm_check(comm)
        assert not counts.any() and not tokens.any() and float(loss) == 0.0
        counts.fill_(5), tokens.fill_(5), loss.fill_(5.0)
    ccl.ccl_comm_destroy(comm)
    assert bool((logits == 1).all())

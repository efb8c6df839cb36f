"""ccl_allreduce_residual_rmsnorm_e4m3 on rows narrower than a warp's columns, many of them and over many ranks, whose
chunks end inside rows: lanes without columns ask for elements behind the last row."""
import pytest
import torch

from test_norm_e4m3 import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [1, 2, 3, 5, 9, 13, 17, 20, 22, 24, 31])
@pytest.mark.parametrize("p, rows, group", [(16, 152, 0), (33, 153, 32), (64, 152, 0), (64, 200, 32)])
def test_narrow_rows(dtype, hidden, p, rows, group):
    run(dtype, p, rows, hidden, group)

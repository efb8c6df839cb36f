"""Lists of thousands of choices a token: the three operators on rows, around the sizes where a list and a kernel's
own arrays together pass the shared memory that a kernel has without asking (48 KB, 16 bytes a choice)."""
import pytest
import torch

from test_expert_rows import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("k", [3008, 3009, 3040, 3071, 4096])
@pytest.mark.parametrize("hidden", [16, 13])
def test_long_lists(k, hidden):
    Layer("bf16", 1, 2, hidden, k).all()


@pytest.mark.parametrize("dtype, p, k", [("f32", 3, 3009), ("f16", 9, 3050)])
def test_long_lists_of_more_ranks(dtype, p, k):
    Layer(dtype, p, 2, 24, k, weighted=False).all()

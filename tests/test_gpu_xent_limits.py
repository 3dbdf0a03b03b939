"""sgemm_xent and sgemm_xent_grad at the ends of their ranges."""
import pytest

from gpu_util import torch_cuda
from test_gpu_xent import check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7])
def test_few_rows_of_a_large_vocabulary(T):
    """A vocabulary whose one row of P would be longer than the K loop takes."""
    torch = torch_cuda()
    check(torch, *problem(torch, T, 17_180_000, 8, torch.bfloat16))

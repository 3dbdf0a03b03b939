"""Operands of more rows than one launch has workgroups for, copied into aligned
rows first."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import assert_equal
from test_gpu_w4 import weight
from test_gpu_w4_forms import product
from test_gpu_xent import check, problem

pytestmark = pytest.mark.gpu

ROWS = (1 << 24) + 321              # of 256 threads each: past 2^32


def small(torch, shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def test_grouped_rows():
    torch = torch_cuda()
    A, B = small(torch, (ROWS, 3), 1, torch.bfloat16), small(torch, (2, 3, 8), 2, torch.bfloat16)
    cut = 5_000_001
    C = lib.sgemm_grouped(A, B, torch.tensor([0, cut, ROWS], dtype=torch.int32, device="cuda"))
    assert_equal(torch, C[:cut], A[:cut].double() @ B[0].double())
    assert_equal(torch, C[cut:], A[cut:].double() @ B[1].double())


def test_weight_gradient_rows():
    torch = torch_cuda()
    A, D = small(torch, (ROWS, 3), 1, torch.bfloat16), small(torch, (ROWS, 5), 2, torch.bfloat16)
    C = lib.sgemm_grouped_wgrad(A, D, torch.tensor([0, 700, ROWS], dtype=torch.int32, device="cuda"))
    # (sums of up to 2^24 products of 9 at most: below 2^24 in every partial sum that random signs give)
    assert_equal(torch, C[1], A[700:].double().T.contiguous() @ D[700:].double())


def test_4bit_product_rows():
    torch = torch_cuda()
    W = weight(torch, 8, 3, 32, True, torch.float16, exact=True)
    X = small(torch, (1 << 24, 3), 3, torch.float16)
    assert_equal(torch, lib.sgemm_w4(X, W), product(torch, X, W))


@pytest.mark.parametrize("T", [2, 40])
def test_vocabulary_rows(T):
    torch = torch_cuda()
    check(torch, *problem(torch, T, ROWS, 3, torch.bfloat16))

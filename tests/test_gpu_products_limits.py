"""Operands of more rows than one launch has workgroups for, copied into aligned
rows first."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import assert_equal, padded
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


@pytest.mark.parametrize("T,N", [(65536, 8192), (65536, 4097), (9_000_000, 40)])
def test_offsets_that_decrease_stay_within_their_operands(T, N):
    """Groups that all overlap have more tiles than 32 bits count; the call
    leaves what lies around C alone, and the next call is right."""
    torch = torch_cuda()
    e, G, K = torch.bfloat16, 65535, 8
    A = small(torch, (T, K), 1, e)
    B = small(torch, (1, K, N), 2, e).expand(G, K, N)
    C = padded(torch, torch.zeros(T, N, dtype=e, device="cuda"), 8, 8, fill=99.0)
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[1::2] = T                                   # 0, T, 0, T, ...
    lib.sgemm_grouped(A, B, off, C=C)
    around = torch.as_strided(C, (T, N + 8), (N + 8, 1))
    assert (around[:, N:] == 99.0).all()
    assert (torch.as_strided(C, (8,), (1,), C.storage_offset() - 8) == 99.0).all()
    off.fill_(T)
    off[:2] = torch.tensor([0, T // 2], dtype=torch.int32)
    lib.sgemm_grouped(A, B, off, C=C)
    ref = A.float() @ B[0].float()                  # (exact: integers)
    assert torch.equal(C, ref.to(e)) and (around[:, N:] == 99.0).all()

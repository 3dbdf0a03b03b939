"""8-bit integers where rounding, layouts and the largest tiles have their limits."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def next_to_halves(torch, top):
    """Rows whose largest magnitudes are `top` [M] (FP32): those, and for each
    odd multiple of half the row's scale the nearest FP32 values to it."""
    s = (top.double() / 127).float().clamp(min=2.0 ** -126).double()
    half = ((torch.arange(-127, 127) + 0.5).double() * s[:, None]).float()
    up, down = (torch.nextafter(half, torch.full_like(half, v)) for v in (float("inf"), -float("inf")))
    x = torch.cat([top[:, None], half, up, down], 1)
    return torch.maximum(torch.minimum(x, top[:, None]), -top[:, None])


@pytest.mark.parametrize("t", ["float32", "bfloat16"])
def test_quantize_with_scales_next_to_the_smallest(t):
    """Scales of 2^-126 to 2^-124, half of which is no normal FP32 value (FP16
    has no rows of such scales): each value is the nearest, halves to even, by
    the quotient in exact arithmetic (Python's fractions round so)."""
    from fractions import Fraction
    torch = torch_cuda()
    t = getattr(torch, t)
    g = torch.Generator().manual_seed(3)
    top = ((torch.rand(60, generator=g) * 3 + 1) * 127).double() * 2.0 ** -126
    x = next_to_halves(torch, top.float().to(t).float()).to(t).float()
    s = (x.abs().amax(1).double() / 127).float().clamp(min=2.0 ** -126)
    got = lib.sgemm_i8_quantize(x.to(t).cuda())
    assert torch.equal(got.scales.cpu(), s)
    want = [[round(Fraction(v) / Fraction(d)) for v in row] for row, d in zip(x.tolist(), s.tolist())]
    assert torch.equal(got.values.cpu().long(), torch.tensor(want))


def test_matrices_of_groups_of_one_row():
    """A group's only row has no row step of its own: rows at equal distances
    are taken as they lie, whatever step their tensor names for that dimension."""
    torch = torch_cuda()
    w = torch.randn(5, 3, 45, generator=torch.Generator().manual_seed(1)).cuda()
    flat = w.view(1, 15, 45).transpose(0, 1)                # [15,1,45], row step 15 * 45
    far = w[:, 1:2]                                         # [5,1,45], 3 * 45 from row to row
    for x in (flat, far, far.clone(), w[:1, :1], w[:0, :1]):
        want = lib.sgemm_i8_quantize(x.reshape(-1, 45))
        got = lib.sgemm_i8_quantize(x)
        assert got.values.shape == x.shape and torch.equal(got.values.view(-1, 45), want.values)
        assert torch.equal(got.scales.view(-1), want.scales)
        # the same 8-bit rows, laid out as x is
        held = torch.zeros(5, 3, 45, dtype=torch.int8, device="cuda").as_strided(x.shape, x.stride())
        held.copy_(got.values)
        assert torch.equal(lib.sgemm_i8_dequantize(lib.I8Matrix(held, got.scales)).view(-1, 45), lib.sgemm_i8_dequantize(want))
    for x in (w[:, :1, ::2], w[:1, :1].expand(4, 1, 45)):   # columns apart; rows on one another
        with pytest.raises((ValueError, lib.SgemmError)):
            lib.sgemm_i8_quantize(x)

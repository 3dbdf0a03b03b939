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

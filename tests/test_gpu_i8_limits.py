"""8-bit integers where rounding, layouts and the largest tiles have their limits."""
import pytest

import fp32_sgemm_tuning_amd as lib
from fp32_sgemm_tuning_amd import capi
from gpu_util import torch_cuda
from test_gpu_i8 import TYPES, check, ints8, laid, product_ref, scales

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


# Tiles of 256 x 256, one workgroup per compute unit (256 of them) taking several:
# two each; 84 and 33 left over, which are cut in two and in four; 164 left over,
# which are not cut.
WIDE = [(8000, 4090), (4900, 4300), (4350, 4300), (5000, 5300)]
# one unit of 128 k, two, three and more; whole, with a remainder, with a cut chunk
UNITS = [0, 16, 100, 128, 129, 255, 272, 384, 400, 2047]


def wide_case(torch, M, N, K):
    x, w = ints8(torch, (M, K), 1), ints8(torch, (N, K), 2)
    sx, sw = scales(torch, M, 3, 0.01), scales(torch, N, 4, 0.01)
    X, W = (x, w) if K == 0 else (laid(torch, x), laid(torch, w))
    return lib.I8Matrix(X, sx), lib.I8Matrix(W, sw), product_ref(x, sx, w, sw)


@pytest.mark.parametrize("M,N", WIDE)
@pytest.mark.parametrize("K", UNITS)
def test_several_tiles_to_a_workgroup(M, N, K):
    torch = torch_cuda()
    X, W, ref = wide_case(torch, M, N, K)
    for t in TYPES:
        check(torch, lib.sgemm_i8(X, W, out_dtype=getattr(torch, t)), ref, what=t)


@pytest.mark.parametrize("M,N", WIDE)
@pytest.mark.parametrize("t", TYPES)
def test_several_tiles_added_to_a_given_result(M, N, t):
    torch = torch_cuda()
    t, K = getattr(torch, t), 272
    X, W, ref = wide_case(torch, M, N, K)
    for off in (0, 3):
        buf = torch.full((M * (N + 5) + 8,), float("nan"), dtype=t, device="cuda")
        C = buf[off:off + M * (N + 5)].view(M, N + 5)[:, :N]
        lib.sgemm_i8(X, W, C)
        check(torch, C, ref)
        start = torch.randn(M, N, generator=torch.Generator().manual_seed(5)).to(t).cuda()
        C.copy_(start)
        lib.sgemm_i8(X, W, C, alpha=-0.5, beta=0.75)
        check(torch, C, -0.5 * ref, 0.75 * start.double())
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[off:off + M * (N + 5)].view(M, N + 5)[:, :N] = False
        assert buf[outside].isnan().all()


# (rows of each group, N): 47 rows of 256 x 256 tiles in six and nine columns; 70
# groups of a tile or two, past the 64 that are counted at once
WIDE_GROUPS = [([3000, 0, 1, 5200, 256, 700, 0, 2049], 1300), ([3000, 0, 1, 5200, 256, 700, 0, 2049], 2100), ([140, 300] * 35, 1100)]


def grouped_case(torch, rows, N, K):
    """Operands, bounds (rows 0 to 2 and the last four are of no group) and the 64-bit products of the groups."""
    off = [3]
    for r in rows:
        off.append(off[-1] + r)
    T, G = off[-1] + 4, len(rows)
    x, w = ints8(torch, (T, K), 1), ints8(torch, (G, N, K), 2)
    sx, sw = scales(torch, T, 3, 0.01), scales(torch, (G, N), 4, 0.01)
    ref = torch.full((T, N), float("nan"), dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(zip(off, off[1:])):
        ref[a:b] = product_ref(x[a:b], sx[a:b], w[g], sw[g])
    return lib.I8Matrix(laid(torch, x), sx), lib.I8Matrix(laid(torch, w), sw), torch.tensor(off, dtype=torch.int32, device="cuda"), ref


@pytest.mark.parametrize("rows,N", WIDE_GROUPS)
@pytest.mark.parametrize("K", [100, 128, 272, 400])
def test_several_tiles_of_groups_to_a_workgroup(rows, N, K):
    torch = torch_cuda()
    X, W, off, ref = grouped_case(torch, rows, N, K)
    for t in TYPES:
        t = getattr(torch, t)
        C = torch.full((ref.shape[0], N + 3), 7.0, dtype=t, device="cuda")[:, :N]
        lib.sgemm_i8_grouped(X, W, off, C)
        check(torch, C[3:-4], ref[3:-4], what=t)
        assert (C[:3] == 7).all() and (C[-4:] == 7).all()
        before = C.clone()
        lib.sgemm_i8_grouped(X, W, off, C, alpha=0.5, beta=2.0)
        check(torch, C[3:-4], 0.5 * ref[3:-4], 2.0 * before[3:-4].double(), what=t)
        assert (C[:3] == 7).all() and (C[-4:] == 7).all()


def test_rows_throughout_a_result_past_32_bits():
    """600001 tokens of 8192 k: of 2344 tiles the workgroups take nine each and the last ones in parts."""
    torch = torch_cuda()
    x = torch.randint(-128, 128, (600001, 8192), dtype=torch.int8, device="cuda")
    sx = torch.rand(600001, device="cuda") + 0.5
    w, sw = ints8(torch, (200, 8192), 2), scales(torch, 200, 4)
    C = lib.sgemm_i8(lib.I8Matrix(x, sx), lib.I8Matrix(w, sw))
    for first in range(0, 600001, 60000):
        at = torch.arange(first, min(first + 60000, 600001), 37, device="cuda")
        check(torch, C[at], product_ref(x[at], sx[at], w, sw))


def test_several_tiles_in_the_race_check_build(monkeypatch):
    """The same with LDS slots poisoned between their last read and their refill."""
    torch = torch_cuda()
    monkeypatch.setattr(capi, "_lib", capi.open_library(capi.POISON_LIB_PATH))
    for (M, N), K in zip(WIDE * 2, (100, 272, 400, 2047, 128, 129, 255, 1024)):
        X, W, ref = wide_case(torch, M, N, K)
        for t in TYPES:
            check(torch, lib.sgemm_i8(X, W, out_dtype=getattr(torch, t)), ref, what=f"{M}x{N}x{K} {t}")
    for (rows, N), K in zip(WIDE_GROUPS, (400, 128, 272)):
        X, W, off, ref = grouped_case(torch, rows, N, K)
        check(torch, lib.sgemm_i8_grouped(X, W, off)[3:-4], ref[3:-4])

"""Products of 8-bit integers, of one weight and grouped, and the matrices in 8
bits and back, against 64-bit forms.

Tolerance of a product: the sum is exact in 32-bit integers and its 64-bit form
exact too; the result takes four roundings to FP32 (the sum, alpha * sx, two
products), with beta two more (beta * C, the addition), and one to its type.  A
factor (1 + 2^-24)^6 is below 1 + 7 * 2^-24."""
import pytest

import fp32_sgemm_tuning_amd as lib
from fp32_sgemm_tuning_amd import capi
from gpu_util import torch_cuda
from products_util import assert_within, replays, u

pytestmark = pytest.mark.gpu

TYPES = ("float32", "bfloat16", "float16")


def ints8(torch, shape, seed, lo=-128, hi=127):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int8).cuda()


def scales(torch, shape, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(shape, generator=g) + 0.5) * size).cuda()


def laid(torch, x, step=16, offset=0, fill=127):
    """x with rows at multiples of `step` bytes and a chunk more, `offset`
    bytes into its allocation, all else `fill` (what lies behind K)."""
    rows, K = x.shape[-2:]
    lead = x.numel() // max(rows * K, 1)
    ld = (K + step - 1) // step * step + step
    buf = torch.full((offset + lead * rows * ld + 64,), fill, dtype=torch.int8, device=x.device)
    view = buf[offset:offset + lead * rows * ld].view(*x.shape[:-2], rows, ld)[..., :K]
    view.copy_(x)
    return view


def smallest(torch, dtype):
    """Half of the smallest step of a type (its values below the normal range are multiples of that step)."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def product_ref(x, sx, w, sw, alpha=1.0):
    return alpha * (x.double() @ w.double().T.contiguous()) * sx.double()[:, None] * sw.double()


def check(torch, got, ref, added=None, what=""):
    big = ref.abs() if added is None else ref.abs() + added.abs()
    ref = ref if added is None else ref + added
    t = got.dtype
    low = smallest(torch, t) + smallest(torch, torch.float32) * 4
    assert_within(torch, got, ref, 7 * 2 ** -24 * big + u(t, torch) * (ref.abs() + 7 * 2 ** -24 * big) + low, what)


# every launch form, edges of tiles and chunks, one to many rows
SHAPES = [(1, 1, 1), (1, 16, 16), (1, 4096, 4096), (2, 5, 17), (3, 33, 127), (16, 100, 128), (16, 6400, 300), (17, 6401, 129),
          (31, 77, 1000), (33, 257, 513), (48, 129, 2047), (49, 64, 64), (64, 6403, 144), (64, 200, 4097), (65, 70, 255),
          (100, 1111, 1024), (128, 8192, 512), (200, 300, 1000), (257, 513, 2047), (300, 4097, 33), (1000, 1024, 8192),
          (1500, 1700, 300), (2500, 2600, 65), (4100, 2100, 100), (3001, 4999, 129), (130, 40000, 272)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("step", [16, 1])
def test_product(M, N, K, step):
    torch = torch_cuda()
    x, w = ints8(torch, (M, K), 1), ints8(torch, (N, K), 2)
    sx, sw = scales(torch, M, 3, 0.01), scales(torch, N, 4, 0.01 * K ** -0.5)
    ref = product_ref(x, sx, w, sw)
    X, W = lib.I8Matrix(laid(torch, x, step), sx), lib.I8Matrix(laid(torch, w, step), sw)
    for t in TYPES:
        got = lib.sgemm_i8(X, W, out_dtype=getattr(torch, t))
        check(torch, got, ref, what=t)
    again = lib.sgemm_i8(X, W, out_dtype=getattr(torch, t))
    assert torch.equal(got, again)
    # one aligned operand and one that is copied; the sums are the same integers
    if step == 1:
        assert torch.equal(lib.sgemm_i8(lib.I8Matrix(laid(torch, x), sx), W), lib.sgemm_i8(X, W))
        assert torch.equal(lib.sgemm_i8(X, lib.I8Matrix(laid(torch, w), sw)), lib.sgemm_i8(X, W))


@pytest.mark.parametrize("M,N", [(1, 40), (20, 70), (40, 40), (64, 100), (70, 300), (600, 700)])
def test_largest_sums(M, N):
    """K at its limit and all values -128: sums of 2^31 - 2^14, in one share of K or several."""
    torch = torch_cuda()
    K = 131071
    x, w = torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    C = lib.sgemm_i8(lib.I8Matrix(laid(torch, x), one[0]), lib.I8Matrix(laid(torch, w), one[1]))
    want = torch.tensor([K * 16384.0, -K * 16256.0], dtype=torch.float64, device="cuda").float()
    assert (C[:, ::2] == want[0]).all() and (C[:, 1::2] == want[1]).all()
    with pytest.raises(lib.SgemmError):
        big = torch.zeros((2, 131072), dtype=torch.int8, device="cuda")
        lib.sgemm_i8(lib.I8Matrix(big, one[0][:1].expand(2).contiguous()), lib.I8Matrix(big, torch.ones(2, device="cuda")))


@pytest.mark.parametrize("M,N,K", [(1, 37, 50), (40, 64, 200), (70, 129, 100), (300, 700, 260), (2300, 2100, 40)])
@pytest.mark.parametrize("t", TYPES)
def test_alpha_beta_and_a_given_result(M, N, K, t):
    torch = torch_cuda()
    t = getattr(torch, t)
    x, w = ints8(torch, (M, K), 1), ints8(torch, (N, K), 2)
    sx, sw = scales(torch, M, 3, 0.02), scales(torch, N, 4, 0.02)
    X, W = lib.I8Matrix(x, sx), lib.I8Matrix(w, sw)
    ref = product_ref(x, sx, w, sw, -1.5)
    for off in (0, 3):
        buf = torch.full((M + 2, N + 5), float("nan"), dtype=t, device="cuda").view(-1)
        C = buf[off:off + M * (N + 5)].view(M, N + 5)[:, :N]
        # beta 0: what C holds is not read
        assert lib.sgemm_i8(X, W, C, alpha=-1.5) is C
        check(torch, C, ref)
        start = torch.randn(M, N, generator=torch.Generator().manual_seed(5)).to(t).cuda()
        C.copy_(start)
        lib.sgemm_i8(X, W, C, alpha=-1.5, beta=0.75)
        check(torch, C, ref, 0.75 * start.double())
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[off:off + M * (N + 5)].view(M, N + 5)[:, :N] = False
        assert buf[outside].isnan().all()


@pytest.mark.parametrize("M", [1, 20, 100, 3000])
def test_scales_of_any_kind(M):
    """A NaN, infinite, zero or tiny scale reaches its row or column alone."""
    torch = torch_cuda()
    N, K = 300, 70
    x, w = ints8(torch, (M, K), 1, 1, 100), ints8(torch, (N, K), 2, 1, 100)
    sx, sw = scales(torch, M, 3), scales(torch, N, 4)
    sx[0], sw[5], sw[6], sw[7], sw[8] = float("nan") if M > 1 else 1.0, float("nan"), float("inf"), 0.0, 1e-38
    C = lib.sgemm_i8(lib.I8Matrix(x, sx), lib.I8Matrix(w, sw))
    rows = slice(1, None) if M > 1 else slice(None)
    if M > 1:
        assert C[0].isnan().all()
    assert C[rows, 5].isnan().all() and (C[rows, 6] == float("inf")).all() and (C[rows, 7] == 0).all()
    keep = [n for n in range(N) if n not in (5, 6)]
    check(torch, C[rows][:, keep], product_ref(x, sx, w, sw)[rows][:, keep])


def test_empty():
    torch = torch_cuda()
    def m(rows, K):
        return lib.I8Matrix(torch.zeros(rows, K, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda"))
    assert lib.sgemm_i8(m(0, 5), m(7, 5)).shape == (0, 7)
    assert lib.sgemm_i8(m(5, 5), m(0, 5)).shape == (5, 0)
    for M in (3, 100, 3000):
        assert (lib.sgemm_i8(m(M, 0), m(2100, 0)) == 0).all()
        C = torch.full((M, 2100), 3.0, device="cuda")
        assert (lib.sgemm_i8(m(M, 0), m(2100, 0), C, beta=0.5) == 1.5).all()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    W = lib.I8Matrix(torch.zeros(3, 6, 5, dtype=torch.int8, device="cuda"), torch.ones(3, 6, device="cuda"))
    assert lib.sgemm_i8_grouped(m(0, 5), W, off).shape == (0, 6)
    q = lib.sgemm_i8_quantize(torch.zeros(0, 5, device="cuda"))
    assert q.values.shape == (0, 5) and q.scales.shape == (0,)
    q = lib.sgemm_i8_quantize(torch.zeros(4, 0, device="cuda"))
    assert q.values.shape == (4, 0) and (q.scales == 2.0 ** -126).all() and lib.sgemm_i8_dequantize(q).shape == (4, 0)


# (rows of each group, N, K)
GROUPS = [([1], 16, 16), ([0, 3, 0, 1, 4], 33, 100), ([8] * 16, 256, 512), ([5, 0, 60, 31, 2], 300, 257), ([100, 0, 250, 1], 129, 130),
          ([500, 700, 3], 511, 96), ([2500, 0, 900, 600], 1300, 200), ([0] * 70 + [40] + [1] * 30, 64, 2047), ([3] * 300, 70, 64)]


@pytest.mark.parametrize("rows,N,K", GROUPS)
@pytest.mark.parametrize("step", [16, 1])
def test_grouped(rows, N, K, step):
    torch = torch_cuda()
    off = [2]                                   # rows 0, 1 and the last three are of no group
    for r in rows:
        off.append(off[-1] + r)
    T, G = off[-1] + 3, len(rows)
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w = ints8(torch, (T, K), 1), ints8(torch, (G, N, K), 2)
    sx, sw = scales(torch, T, 3, 0.01), scales(torch, (G, N), 4, 0.01)
    X, W = lib.I8Matrix(laid(torch, x, step), sx), lib.I8Matrix(laid(torch, w, step), sw)
    for t in TYPES:
        C = torch.full((T, N), 7.0, dtype=getattr(torch, t), device="cuda")
        lib.sgemm_i8_grouped(X, W, dev, C, alpha=0.5)
        for g, (a, b) in enumerate(zip(off, off[1:])):
            check(torch, C[a:b], product_ref(x[a:b], sx[a:b], w[g], sw[g], 0.5), what=f"group {g}")
        assert (C[:2] == 7).all() and (C[-3:] == 7).all()
        before = C.clone()
        lib.sgemm_i8_grouped(X, W, dev, C, alpha=0.5, beta=2.0)
        for g, (a, b) in enumerate(zip(off, off[1:])):
            check(torch, C[a:b], product_ref(x[a:b], sx[a:b], w[g], sw[g], 0.5), 2.0 * before[a:b].double(), what=f"group {g}")
    # the scales of the groups further apart than one after another
    far = torch.full((G, N + 9), float("nan"), device="cuda")
    far[:, :N] = sw
    a = lib.sgemm_i8_grouped(X, lib.I8Matrix(W.values, far[:, :N]), dev)
    b = lib.sgemm_i8_grouped(X, W, dev)
    assert torch.equal(a[2:-3], b[2:-3])


@pytest.mark.parametrize("rows", [4, 100, 2000])
def test_bounds_that_are_out_of_range(rows):
    """Bounds behind the rows, or below 0, are taken as the nearest row."""
    torch = torch_cuda()
    x, w = ints8(torch, (rows, 48), 1), ints8(torch, (2, 70, 48), 2)
    sx, sw = scales(torch, rows, 3), scales(torch, (2, 70), 4)
    dev = torch.tensor([-5, rows // 2, rows + 1000], dtype=torch.int32, device="cuda")
    C = lib.sgemm_i8_grouped(lib.I8Matrix(x, sx), lib.I8Matrix(w, sw), dev)
    check(torch, C[:rows // 2], product_ref(x[:rows // 2], sx[:rows // 2], w[0], sw[0]))
    check(torch, C[rows // 2:], product_ref(x[rows // 2:], sx[rows // 2:], w[1], sw[1]))


def quant_ref(torch, x):
    """Scales and values by the definition, in 64 bits on the CPU."""
    x = x.cpu()
    top = x.float().abs().amax(-1) if x.shape[-1] else torch.zeros(x.shape[:-1])
    s = (top.double() / 127).float().clamp(min=2.0 ** -126)             # a division rounded once to FP32
    return s, torch.round(x.double() / s.double()[..., None])


@pytest.mark.parametrize("M,K", [(1, 1), (3, 5), (17, 1001), (4, 8), (9, 64), (5, 1024), (6, 1025), (3, 4096), (2, 4097), (3, 10000), (300, 2047)])
@pytest.mark.parametrize("t", TYPES)
def test_quantize(M, K, t):
    torch = torch_cuda()
    t = getattr(torch, t)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M + K)).to(t)
    x[0] *= 0
    if M > 1:
        x[1, 0] = 100.0
    s, q = quant_ref(torch, x)
    for off in (0, 1):
        buf = torch.full((off + M * (K + 3) + 8,), float("nan"), dtype=t, device="cuda")
        X = buf[off:off + M * (K + 3)].view(M, K + 3)[:, :K]
        X.copy_(x)
        got = lib.sgemm_i8_quantize(X)
        assert torch.equal(got.scales.cpu(), s)
        assert torch.equal(got.values.cpu().double(), q)
        back = lib.sgemm_i8_dequantize(got, t)
        assert torch.equal(back.cpu(), (q * s.double()[:, None]).float().to(t))     # q * s rounded to FP32, then to t
    assert torch.equal(lib.sgemm_i8_dequantize(got).cpu(), (q * s.double()[:, None]).float())


@pytest.mark.parametrize("t", TYPES)
def test_quantize_next_to_the_borders(t):
    """Values half-way between two steps and next to that: every odd multiple
    of half a scale that is a value of the type, and its neighbours."""
    torch = torch_cuda()
    t = getattr(torch, t)
    g = torch.Generator().manual_seed(9)
    tops = torch.cat([torch.tensor([127.0, 1.0, 254.0, 63.5, 2.0 ** -10, 381.0]), torch.rand(250, generator=g) * 200 + 0.01]).to(t)
    s = (tops.double() / 127).float().double()
    half = ((torch.arange(-127, 127) + 0.5).double() * s[:, None]).to(t)
    up, down = torch.nextafter(half, torch.full_like(half, float("inf"))), torch.nextafter(half, torch.full_like(half, -float("inf")))
    x = torch.cat([tops[:, None], half, up, down], 1)
    x = torch.maximum(torch.minimum(x, tops[:, None]), -tops[:, None])
    ref_s, q = quant_ref(torch, x)
    got = lib.sgemm_i8_quantize(x.cuda())
    assert torch.equal(got.scales.cpu(), ref_s)
    assert torch.equal(got.values.cpu().double(), q)


def test_quantize_small_and_not_finite():
    torch = torch_cuda()
    x = torch.randn(8, 700, generator=torch.Generator().manual_seed(1))
    x[1] *= 1e-37
    x[2] *= 1e-41
    x[3] *= 1e38 / 10
    x[4, 699] = float("nan")
    x[5, 3] = float("inf")
    x[6, 4] = -float("inf")
    x[7] = torch.finfo(torch.float32).max
    got = lib.sgemm_i8_quantize(x.cuda())
    rows = [0, 1, 2, 3, 7]
    s, q = quant_ref(torch, x[rows])
    assert torch.equal(got.scales.cpu()[rows], s) and torch.equal(got.values.cpu()[rows].double(), q)
    assert got.scales[4:7].isnan().all() and (got.values[4:7] == 0).all()
    assert lib.sgemm_i8_dequantize(got)[4:7].isnan().all()
    y = lib.sgemm_i8(got, lib.sgemm_i8_quantize(torch.ones(40, 700, device="cuda")))
    assert y[4:7].isnan().all() and not y[:4].isnan().any()


def test_matrices_of_groups():
    """Three-dimensional matrices are quantised as their rows are."""
    torch = torch_cuda()
    w = torch.randn(3, 10, 45, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    W = lib.sgemm_i8_quantize(w)
    flat = lib.sgemm_i8_quantize(w.view(30, 45))
    assert torch.equal(W.values, flat.values.view(3, 10, 45)) and torch.equal(W.scales, flat.scales.view(3, 10))
    assert torch.equal(lib.sgemm_i8_dequantize(W), lib.sgemm_i8_dequantize(flat).view(3, 10, 45))
    with pytest.raises(ValueError):
        lib.sgemm_i8_quantize(torch.zeros(4, 20, 45, device="cuda")[:, :10])


@pytest.mark.parametrize("shape", [(3, 0, 8), (3, 5, 0), (3, 1, 0), (0, 5, 8), (3, 0, 0)])
def test_empty_matrices_of_groups(shape):
    torch = torch_cuda()
    W = lib.sgemm_i8_quantize(torch.empty(shape, device="cuda"))
    assert W.values.shape == shape and torch.equal(W.scales, torch.full(shape[:2], 2.0 ** -126, device="cuda"))
    assert lib.sgemm_i8_dequantize(W).shape == shape


@pytest.mark.parametrize("M", [1, 40, 300])
def test_quantised_product_of_float_rows(M):
    """Quantise, multiply: off from the product of the floats by what the
    quantisation may be off, half a step of each factor's row."""
    torch = torch_cuda()
    N, K = 200, 999
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).cuda()
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(2)) * K ** -0.5).bfloat16().cuda()
    X, W = lib.sgemm_i8_quantize(x), lib.sgemm_i8_quantize(w)
    C = lib.sgemm_i8(X, W)
    hx, hw = X.scales.double()[:, None] / 2, W.scales.double()[:, None] / 2
    bound = x.double().abs() @ hw.expand(N, K).T.contiguous() + hx.expand(M, K) @ (w.double().abs() + hw).T.contiguous()
    ref = x.double() @ w.double().T.contiguous()
    assert ((C.double() - ref).abs() <= bound * (1 + 2 ** -20) + 8 * 2 ** -24 * (ref.abs() + bound)).all()


@pytest.mark.parametrize("M,N,K,step", [(1, 512, 300, 16), (40, 300, 200, 1), (100, 500, 8192, 16), (700, 800, 96, 16)])
def test_graph(M, N, K, step):
    torch = torch_cuda()
    x, w = laid(torch, ints8(torch, (M, K), 1), step), laid(torch, ints8(torch, (N, K), 2), step)
    sx, sw = scales(torch, M, 3), scales(torch, N, 4)
    X, W = lib.I8Matrix(x, sx), lib.I8Matrix(w, sw)
    f = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)

    def run():
        q = lib.sgemm_i8_quantize(f)
        return [lib.sgemm_i8(X, W), lib.sgemm_i8(q, W, out_dtype=torch.bfloat16)]

    def refresh(i):
        x.copy_(ints8(torch, (M, K), 10 + i))
        f.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(20 + i)))

    def checked(outs, i):
        check(torch, outs[0], product_ref(x, sx, w, sw), what=f"replay {i}")
        assert torch.equal(outs[1], run()[1])
    replays(torch, run, lambda o: o, refresh, checked)


def test_two_streams_and_a_given_one():
    torch = torch_cuda()
    x, w = ints8(torch, (100, 8192), 1), ints8(torch, (600, 8192), 2)
    X, W = lib.I8Matrix(x, scales(torch, 100, 3)), lib.I8Matrix(w, scales(torch, 600, 4))
    want = lib.sgemm_i8(X, W)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[lib.sgemm_i8(X, W, stream=s) for s in streams] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for row in got for g in row)


@pytest.mark.parametrize("offset", range(8))
def test_few_rows_at_any_byte(offset):
    """Rows of any alignment, the last ending with its allocation's last byte."""
    torch = torch_cuda()
    M, N, K = 3, 50, 143 + offset
    x, w = ints8(torch, (M, K), 1), ints8(torch, (N, K), 2)
    sx, sw = scales(torch, M, 3), scales(torch, N, 4)
    far = torch.full((offset + N * K,), 99, dtype=torch.int8, device="cuda")
    far[offset:].view(N, K).copy_(w)
    got = lib.sgemm_i8(lib.I8Matrix(x, sx), lib.I8Matrix(far[offset:].view(N, K), sw))
    check(torch, got, product_ref(x, sx, w, sw))
    near = torch.full((offset + M * K,), 99, dtype=torch.int8, device="cuda")
    near[offset:].view(M, K).copy_(x)
    assert torch.equal(lib.sgemm_i8(lib.I8Matrix(near[offset:].view(M, K), sx), lib.I8Matrix(w, sw)), got)


def test_past_32_bits():
    """Operands and results of more than 2^32 bytes; the last rows lie behind."""
    torch = torch_cuda()
    w = torch.randint(-128, 128, (600001, 8192), dtype=torch.int8, device="cuda")
    sw = torch.rand(600001, device="cuda") + 0.5
    for M in (1, 40, 200):
        x = ints8(torch, (M, 8192), M)
        sx = scales(torch, M, 3)
        C = lib.sgemm_i8(lib.I8Matrix(x, sx), lib.I8Matrix(w, sw))
        check(torch, C[:, -300:], product_ref(x, sx, w[-300:], sw[-300:]))
    # the same memory as the tokens, and as the groups' weights
    C = lib.sgemm_i8(lib.I8Matrix(w, sw), lib.I8Matrix(x, sx), out_dtype=torch.bfloat16)
    check(torch, C[-300:], product_ref(w[-300:], sw[-300:], x, sx))
    del C
    G = w[:600000].view(4, 150000, 8192)
    dev = torch.tensor([0, 10, 20, 30, 200], dtype=torch.int32, device="cuda")
    C = lib.sgemm_i8_grouped(lib.I8Matrix(x, sx), lib.I8Matrix(G, sw[:600000].view(4, -1)), dev)
    check(torch, C[30:, -300:], product_ref(x[30:], sx[30:], G[3, -300:], sw[599700:600000]))


def test_race_check_build(monkeypatch):
    """The same products with LDS stages poisoned between their last read and
    their refill."""
    torch = torch_cuda()
    monkeypatch.setattr(capi, "_lib", capi.open_library(capi.POISON_LIB_PATH))
    for M, N, K in ((70, 300, 1000), (200, 4000, 513), (130, 2000, 8192), (1500, 1700, 300), (4100, 2100, 2047), (3000, 5000, 1024)):
        x, w = ints8(torch, (M, K), 1), ints8(torch, (N, K), 2)
        one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        C = lib.sgemm_i8(lib.I8Matrix(laid(torch, x), one[0]), lib.I8Matrix(laid(torch, w), one[1]))
        assert torch.equal(C, (x.double() @ w.double().T.contiguous()).float())
        dev = torch.tensor([0, M // 3, M // 2, M], dtype=torch.int32, device="cuda")
        w3 = torch.stack([w[:N // 2], w[-(N // 2):], w[1:N // 2 + 1]])
        W = lib.I8Matrix(laid(torch, w3), torch.ones(3, N // 2, device="cuda"))
        C = lib.sgemm_i8_grouped(lib.I8Matrix(laid(torch, x), one[0]), W, dev)
        for g, (a, b) in enumerate(zip(dev.tolist(), dev.tolist()[1:])):
            assert torch.equal(C[a:b], (x[a:b].double() @ w3[g].double().T.contiguous()).float())


def test_refusals():
    torch = torch_cuda()
    def m(shape, dtype=torch.int8):
        return lib.I8Matrix(torch.zeros(shape, dtype=dtype, device="cuda"), torch.ones(shape[:-1], device="cuda"))
    X, W, G = m((6, 8)), m((16, 8)), m((2, 16, 8))
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    for bad in (dict(X=m((6, 8), torch.uint8)), dict(W=lib.I8Matrix(W.values, W.scales.half())), dict(out_dtype=torch.float64),
                dict(C=torch.ones(6, 16, dtype=torch.int32, device="cuda")), dict(C=torch.ones(6, 16, device="cuda"), out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            lib.sgemm_i8(**{**dict(X=X, W=W), **bad})
    for bad in (dict(W=m((16, 9))), dict(W=G), dict(X=lib.I8Matrix(X.values, W.scales)), dict(X=lib.I8Matrix(X.values.cpu(), X.scales)),
                dict(X=lib.I8Matrix(X.values, X.scales.cpu())), dict(beta=1.0), dict(C=torch.ones(5, 16, device="cuda")),
                dict(C=torch.ones(16, 6, device="cuda").T), dict(W=lib.I8Matrix(W.values, torch.ones(32, device="cuda")[::2])),
                dict(X=lib.I8Matrix(torch.zeros(8, 6, dtype=torch.int8, device="cuda").T, X.scales))):
        with pytest.raises(ValueError):
            lib.sgemm_i8(**{**dict(X=X, W=W), **bad})
    for bad in (dict(W=W), dict(offsets=off[:2]), dict(offsets=off.cpu()), dict(offsets=off[None]), dict(X=m((6, 9))), dict(beta=1.0)):
        with pytest.raises(ValueError):
            lib.sgemm_i8_grouped(**{**dict(X=X, W=G, offsets=off), **bad})
    with pytest.raises(TypeError):
        lib.sgemm_i8_grouped(X, G, off.long())
    with pytest.raises(ValueError):
        lib.sgemm_i8_quantize(torch.zeros(8, 6, device="cuda").T)

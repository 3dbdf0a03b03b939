"""4-bit weights: the product against 64 bits, and the way into and out of
the packed form against its definition."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import assert_equal, assert_within, ints, normal, padded, replays, u, w4_values

pytestmark = pytest.mark.gpu


def weight(torch, N, K, group, zeros, dtype, seed=0, exact=False):
    """A random W4Weight; exact: scales that are powers of two."""
    g = torch.Generator().manual_seed(seed)
    Kp = (K + 127) // 128 * 128
    packed = torch.randint(0, 256, (N, Kp // 2), generator=g, dtype=torch.uint8)
    if exact:
        scales = 2.0 ** torch.randint(-2, 2, (N, Kp // group), generator=g)
    else:
        scales = (torch.rand(N, Kp // group, generator=g) + 0.5) * 0.05
    z = torch.randint(0, 16, (N, Kp // group), generator=g, dtype=torch.uint8).cuda() if zeros else None
    return lib.W4Weight(packed.cuda(), scales.to(dtype).cuda(), z, K, group)


FORMS = [(32, True, "bfloat16"), (64, False, "float16"), (128, True, "float16"), (128, False, "bfloat16"),
         (32, False, "float16"), (64, True, "bfloat16")]


@pytest.mark.parametrize("group,zeros,dtype", FORMS)
@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("N,K", [(16, 128), (1, 1), (50, 37), (130, 384), (257, 1000), (64, 2049)])
def test_exact(M, N, K, group, zeros, dtype):
    """Integer X and scales 2^-2 .. 2: every sum of x * (16 + q), of x, and of
    the scaled groups is a multiple of 1/4 below 2^22, so FP32 holds it."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    W = weight(torch, N, K, group, zeros, dtype, seed=N + K, exact=True)
    X = ints(torch, (M, K), -3, 3, dtype, 5)
    q, s = w4_values(torch, W)
    ref = X.double() @ (q * s).T.contiguous()
    assert_equal(torch, lib.sgemm_w4(X, W), ref)
    assert_equal(torch, lib.sgemm_w4(X, W, out_dtype=dtype), ref)


@pytest.mark.parametrize("group,zeros,dtype", FORMS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 300, 8192), (48, 1000, 1024), (200, 515, 520), (1030, 700, 1096)])
def test_against_bound(M, N, K, group, zeros, dtype):
    """Per group the sums of |x| (16 + q) and of |x|, the latter times 16 + z
    at most 31, each off by `group` steps of 2^-23, then scaled and summed
    over K / group groups."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    W = weight(torch, N, K, group, zeros, dtype, seed=1)
    X = normal(torch, (M, K), dtype, 6)
    q, s = w4_values(torch, W)
    ref = X.double() @ (q * s).T.contiguous()
    big = X.double().abs() @ s.T.contiguous()
    tol = 62 * (group + K / group + 4) * 2.0 ** -23 * big
    got = lib.sgemm_w4(X, W)
    assert_within(torch, got, ref, tol)
    # rounding errors are independent: their root sum of squares is far below the bound
    assert ((got.double() - ref).norm() / ref.norm()).item() < 1e-6
    assert_within(torch, lib.sgemm_w4(X, W, out_dtype=dtype), ref, tol + 1.01 * u(dtype, torch) * ref.abs() + 2 ** -25)


@pytest.mark.parametrize("M", [3, 90])
@pytest.mark.parametrize("pad,base,out", [(8, 0, "float32"), (3, 0, "float16"), (8, 8, "float16"), (0, 1, "float32")])
def test_strides_alpha_beta(M, pad, base, out):
    torch = torch_cuda()
    W = weight(torch, 70, 200, 64, True, torch.float16, exact=True)
    X, C0 = ints(torch, (M, 200), -3, 3, torch.float16, 1), ints(torch, (M, 70), -8, 8, getattr(torch, out), 2)
    Xv, Cv = padded(torch, X, pad, base), padded(torch, C0, 5, base, fill=99.0)
    lib.sgemm_w4(Xv, W, C=Cv, alpha=0.5, beta=-2.0)
    q, s = w4_values(torch, W)
    assert_equal(torch, Cv, 0.5 * (X.double() @ (q * s).T.contiguous()) - 2 * C0.double())
    assert (torch.as_strided(Cv, (M, 75), (75, 1))[:, 70:] == 99.0).all()
    Cn = torch.full((M, 70), float("nan"), device="cuda")
    lib.sgemm_w4(Xv, W, C=Cn)
    assert not Cn.isnan().any()


def test_no_inner_extent():
    torch = torch_cuda()
    W = weight(torch, 5, 0, 32, False, torch.bfloat16)
    C = torch.full((2, 5), 3.0, device="cuda")
    lib.sgemm_w4(torch.empty(2, 0, dtype=torch.bfloat16, device="cuda"), W, C=C, beta=2.0)
    assert (C == 6).all()
    assert lib.sgemm_w4_quantize(torch.empty(5, 0, dtype=torch.bfloat16, device="cuda")).packed.shape == (5, 0)


def test_nan_stays_in_its_row():
    torch = torch_cuda()
    for M in (4, 100):
        W = weight(torch, 40, 256, 64, False, torch.bfloat16, exact=True)
        X = ints(torch, (M, 256), -3, 3, torch.bfloat16, 1)
        q, s = w4_values(torch, W)
        ref = X.double() @ (q * s).T.contiguous()
        X[2, 7] = float("nan")
        got = lib.sgemm_w4(X, W)
        keep = torch.arange(M, device="cuda") != 2
        assert got[2].isnan().all()
        assert_equal(torch, got[keep], ref[keep])


def definition(torch, W, group, zeros):
    """q - z, s and z of the definition in 64 bits, element by element."""
    N, K = W.shape
    pad = (-K) % 128
    w = torch.nn.functional.pad(W.double(), (0, pad)).view(N, -1, group)
    lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
    s = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7).float().to(W.dtype).double()
    step = torch.where(s == 0, 1.0, s)
    z = torch.round(-lo / step).clamp(0, 15) if zeros else torch.full_like(lo, 8)
    z = torch.where(s == 0, 0.0 if zeros else 8.0, z)
    q = (torch.round(w / step[..., None]) + z[..., None]).clamp(0, 15)
    q = torch.where((s == 0)[..., None], z[..., None], q)
    return (q - z[..., None]).view(N, -1)[:, :K], s, z


@pytest.mark.parametrize("group,zeros,dtype", FORMS)
@pytest.mark.parametrize("N,K", [(1, 1), (3, 128), (40, 1000), (7, 129), (100, 2048), (333, 37)])
def test_quantize_and_back(N, K, group, zeros, dtype):
    """q follows the definition (w / s rounds the same in FP32 and 64 bits
    unless it lies within 2^-23 of a half, where either neighbour is right)."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    w = normal(torch, (N, K), dtype, N + K, 0.1)
    if K > 64:
        w[0, :64] = 0                                  # a group of zeros
        w[-1, :64] = w[-1, :64].abs() + 1              # one that lies to one side
    W = lib.sgemm_w4_quantize(w, group=group, zeros=zeros)
    qz, s, z = definition(torch, w, group, zeros)
    got, scale = w4_values(torch, W)
    assert_equal(torch, W.scales, s)
    if zeros:
        assert torch.equal(W.zeros.double(), z)
    k = torch.arange(K, device="cuda") // group
    ratio = w.double() / torch.where(s == 0, 1.0, s)[:, k]
    tie = ((ratio - torch.floor(ratio)) - 0.5).abs() < 2.0 ** -20
    assert ((got == qz) | (tie & ((got - qz).abs() == 1))).all()
    back = lib.sgemm_w4_dequantize(W)
    assert back.dtype == dtype and back.shape == (N, K)
    assert_equal(torch, back, got * scale)
    # never further off than half a step of the scale (one where z was rounded), but for s's own rounding of the ends
    err, sk = (back.double() - w.double()).abs(), s[:, k]
    assert (err <= (1.5 if zeros else 0.5) * sk + 8 * u(dtype, torch) * sk * 15).all()


def test_quantize_strides_ties_and_extremes():
    torch = torch_cuda()
    w = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    w[0, :8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -7.0, 3.0])          # s = 1: halves to even
    w[1, 5], w[2, 200] = float("inf"), float("nan")
    w[3] = 6e-8                                                                   # s rounds to 0 in fp16
    for view in (w, padded(torch, w, 8), padded(torch, w, 3, 1)):
        W = lib.sgemm_w4_quantize(view, group=32)
        q, _ = w4_values(torch, W)
        assert q[0, :8].tolist() == [7, 0, 2, 2, 0, -2, -7, 3]
        assert W.scales[1].isnan().tolist() == [True] + [False] * 7
        assert W.scales[2].isnan().tolist() == [False] * 6 + [True, False]
        assert (W.scales[3] == 0).all() and (q[3] == 0).all()
        back = lib.sgemm_w4_dequantize(W)
        assert back[1, :32].isnan().all() and (back[1, 32:] == 0).all() and (back[3] == 0).all()
    Z = lib.sgemm_w4_quantize(w, group=32, zeros=True)
    assert (Z.zeros[3] == 0).all() and Z.scales[1, 0].isnan() and not Z.scales[0].isnan().any()


def test_captured():
    torch = torch_cuda()
    w, X = normal(torch, (300, 520), torch.bfloat16, 1, 0.1), normal(torch, (9, 520), torch.bfloat16, 2)
    many = normal(torch, (200, 520), torch.bfloat16, 3)

    def run():
        W = lib.sgemm_w4_quantize(w, group=64, zeros=True)
        return lib.sgemm_w4(X, W), lib.sgemm_w4(many, W), lib.sgemm_w4_dequantize(W)

    def refresh(i):
        for t, k in ((w, 4), (X, 5), (many, 6)):
            t.copy_(normal(torch, t.shape, t.dtype, 10 * i + k, 0.5))

    def see(outs, i):
        for a, b in zip(outs, run()):
            assert torch.equal(a, b), f"replay {i}"
    replays(torch, run, lambda o: o, refresh, see)


def test_refusals():
    torch = torch_cuda()
    W = weight(torch, 6, 256, 64, True, torch.bfloat16)
    X = torch.ones(3, 256, dtype=torch.bfloat16, device="cuda")
    for X2, W2 in ((X.half(), W), (X.float(), W), (X, W._replace(scales=W.scales.float())),
                   (X, W._replace(packed=W.packed.int())), (X, W._replace(zeros=W.zeros.int()))):
        with pytest.raises(TypeError):
            lib.sgemm_w4(X2, W2)
    for X2, W2 in ((X[:, :128], W), (X[0], W), (X, W._replace(group=16)), (X, W._replace(K=100)), (X.cpu(), W),
                   (X, W._replace(scales=W.scales[:, :2])), (X, W._replace(zeros=W.zeros.cpu())),
                   (X, W._replace(packed=W.packed[:, ::2]))):
        with pytest.raises(ValueError):
            lib.sgemm_w4(X2, W2)
    with pytest.raises(ValueError):
        lib.sgemm_w4_quantize(X, group=100)
    with pytest.raises(TypeError):
        lib.sgemm_w4_quantize(X.float())
    with pytest.raises(ValueError):
        lib.sgemm_w4(X, W, beta=1.0)
    buf = torch.zeros(6 * 128 + 8, dtype=torch.uint8, device="cuda")
    with pytest.raises(lib.SgemmError):                 # packed rows off a 16-byte boundary
        lib.sgemm_w4(X, W._replace(packed=buf[8:].view(6, 128)))

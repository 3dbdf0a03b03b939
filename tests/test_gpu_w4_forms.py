"""Every launch form of the products with 4-bit weights: groups, zero points,
types, tails of K, strides, alpha and beta, infinities, rounding, and the race
check."""
import pytest

import fp32_sgemm_tuning_amd as lib
from fp32_sgemm_tuning_amd import capi
from gpu_util import torch_cuda
from products_util import assert_equal, assert_within, ints, normal, padded
from test_gpu_w4 import FORMS as KINDS, weight
from w4_forms import SHAPES

pytestmark = pytest.mark.gpu


def values(torch, W):
    """q - z and s of a W4Weight as 64-bit [N,K] arrays, on the device."""
    K, dev = W.K, W.packed.device
    k = torch.arange(K, device=dev)
    word = k // 128 * 16 + 4 * (k % 32 // 8) + k % 128 // 32
    bit = 4 * (k % 8 // 2) + 16 * (k % 2)
    q = (W.packed.view(torch.int32)[:, word] >> bit) & 15
    z = 8 if W.zeros is None else W.zeros[:, k // W.group].int()
    return (q - z).double(), W.scales[:, k // W.group].double()


def product(torch, X, W):
    q, s = values(torch, W)
    return X.double() @ (q * s).T.contiguous()


@pytest.mark.parametrize("group,zeros,dtype", KINDS)
@pytest.mark.parametrize("form,M,N", SHAPES)
def test_exact(form, M, N, group, zeros, dtype):
    """Integer X and scales 2^-2 .. 2: every sum of x * (16 + q), of x and of
    x * (q - z) and of the scaled groups is a multiple of 1/4 below 2^22, so FP32
    holds it.  K is whole chunks or fewer, ends inside a group, and is not a
    multiple of 8 (then X is copied into padded rows)."""
    torch = torch_cuda()
    assert capi.sgemm_w4_select_form(M, N) == form
    dtype = getattr(torch, dtype)
    for K in (40, 384, 517, 1000, 2049):
        W = weight(torch, N, K, group, zeros, dtype, seed=N + K, exact=True)
        X = ints(torch, (M, K), -3, 3, dtype, 5)
        ref = product(torch, X, W)
        assert_equal(torch, lib.sgemm_w4(X, W), ref, f"K {K}")
        assert_equal(torch, lib.sgemm_w4(X, W, out_dtype=dtype), ref, f"K {K}, 16-bit result")


@pytest.mark.parametrize("out", ["float32", "float16"])
@pytest.mark.parametrize("form,M,N", SHAPES)
def test_strides_alpha_beta(form, M, N, out):
    torch = torch_cuda()
    K = 200
    W = weight(torch, N, K, 64, True, torch.float16, exact=True)
    X, C0 = ints(torch, (M, K), -3, 3, torch.float16, 1), ints(torch, (M, N), -8, 8, getattr(torch, out), 2)
    for pad, base in ((8, 8), (3, 1)):
        Xv, Cv = padded(torch, X, pad, base), padded(torch, C0, 5, base, fill=99.0)
        lib.sgemm_w4(Xv, W, C=Cv, alpha=0.5, beta=-2.0)
        assert_equal(torch, Cv, 0.5 * product(torch, X, W) - 2 * C0.double())
        assert (torch.as_strided(Cv, (M, N + 5), (N + 5, 1))[:, N:] == 99.0).all()


@pytest.mark.parametrize("group,zeros,dtype", KINDS)
@pytest.mark.parametrize("form,M,N", SHAPES)
def test_infinities_and_values_near_the_end(form, M, N, group, zeros, dtype):
    """An infinity gives what the formula gives (infinities of q - z's sign, NaN
    where q is z), a NaN a row of NaN, and BF16 values whose product with 16 + q
    passes FP32's range the number they stand for; other rows keep theirs."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    K = 520
    W = weight(torch, N, K, group, zeros, dtype, seed=N, exact=True)
    X = ints(torch, (M, K), -3, 3, dtype, 5)
    special = [(7, float("inf")), (K - 1, -float("inf")), (130, float("nan")), (300, float("inf"))]
    if dtype == torch.bfloat16:
        special += [(11, 2.0 ** 124), (400, -(2.0 ** 124))]
    for i, (k, v) in enumerate(special):
        if M <= len(special):                             # one of them in the last row, as seen from the seed
            i = M - 1
            k, v = special[(N + group) % len(special)]
        row = i * ((M - 1) // len(special) or 1)
        if abs(v) < float("inf"):
            X[row] = 0                                    # (one term: exact)
        X[row, k] = v
    ref = product(torch, X, W)
    got = lib.sgemm_w4(X, W)
    assert not ref.isfinite().all() or dtype == torch.bfloat16
    assert torch.equal(got.isnan(), ref.isnan())
    live = ~ref.isnan()
    assert_equal(torch, got[live], ref[live])


@pytest.mark.parametrize("group,zeros,dtype", [k for k in KINDS if k[0] < 128])
@pytest.mark.parametrize("form,M,N", SHAPES)
def test_what_lies_behind_K_is_not_used(form, M, N, group, zeros, dtype):
    """The last chunk's values, scales and zero points behind K may hold
    anything."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    for K in (8, 129, 264, 351):
        W = weight(torch, N, K, group, zeros, dtype, seed=K, exact=True)
        X = ints(torch, (M, K), -3, 3, dtype, 5)
        ref = product(torch, X, W)
        used = (K + group - 1) // group
        W.scales[:, used:] = float("nan")
        if zeros:
            W.zeros[:, used:] = 255
        got = lib.sgemm_w4(X, W)
        assert_equal(torch, got, ref, f"K {K}")
        assert_equal(torch, lib.sgemm_w4_dequantize(W), (lambda q, s: q * s)(*values(torch, W)))
        X[0, 0] = float("inf")
        want, got = product(torch, X, W)[0], lib.sgemm_w4(X, W)[0]
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~want.isnan()].double(), want[~want.isnan()])


@pytest.mark.parametrize("group,zeros,dtype", KINDS)
@pytest.mark.parametrize("form,M,N", SHAPES)
def test_inputs_of_one_sign(form, M, N, group, zeros, dtype):
    """Sums of x * (16 + q) and 16 + z times the sum of x, which grow with K where
    X has one sign, cancel: their FP32 steps remain (31 times |x| each, `group`
    sums; then one per scaled group).  The tiles sum x * (q - z), 15 times |x| at
    most."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    K = 1096
    W = weight(torch, N, K, group, zeros, dtype, seed=N)
    X = normal(torch, (M, K), dtype, 6).abs()
    q, s = values(torch, W)
    tol = (15 if form >= 6 else 62) * (group + K / group + 4) * 2.0 ** -23 * (X.double() @ s.T.contiguous())
    assert_within(torch, lib.sgemm_w4(X, W), X.double() @ (q * s).T.contiguous(), tol)


def test_race_check_build(monkeypatch):
    """The tiles' two stages of X poisoned between their last read and their
    refill."""
    torch = torch_cuda()
    monkeypatch.setattr(capi, "_lib", capi.open_library(capi.POISON_LIB_PATH))
    for form, M, N in SHAPES:
        if form < 6:
            continue
        for group, zeros, dtype in KINDS:
            W = weight(torch, N, 1000, group, zeros, getattr(torch, dtype), seed=N, exact=True)
            X = ints(torch, (M, 1000), -3, 3, getattr(torch, dtype), 5)
            assert_equal(torch, lib.sgemm_w4(X, W), product(torch, X, W), f"{M} x {N}, groups of {group}")

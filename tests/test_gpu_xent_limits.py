"""sgemm_xent and sgemm_xent_grad at the ends of their ranges."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import assert_within, ints, replays, u, xent_ref
from test_gpu_xent import check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7])
def test_few_rows_of_a_large_vocabulary(T):
    """A vocabulary whose one row of P would be longer than the K loop takes."""
    torch = torch_cuda()
    check(torch, *problem(torch, T, 17_180_000, 8, torch.bfloat16))


def spread(torch, T, V, H, shift, decades, seed):
    """Integer X and W (so that logits are exact), W off centre by `shift`,
    FP16; row weights over `decades` decades up to 2^12, far above the steps
    that FP16 gradients end in."""
    X, W = ints(torch, (T, H), -3, 3, torch.float16, seed), ints(torch, (V, H), shift - 3, shift + 3, torch.float16, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    target = torch.randint(0, V, (T,), generator=g).cuda()
    dloss = 2.0 ** 12 * 10.0 ** (-decades * torch.arange(T) / max(T - 1, 1))
    return X, W, target, dloss[torch.randperm(T, generator=g)].cuda()


@pytest.mark.parametrize("T,V,H,alpha,shift,decades", [
    (64, 32000, 64, 0.125, 0, 6), (64, 32000, 64, 0.125, 0, 12), (512, 50021, 72, 0.0625, 0, 6), (300, 129, 61, 0.125, 0, 9),
    (64, 128000, 64, 2.0 ** -10, 6, 6), (20, 20011, 64, 2.0 ** -10, 6, 6), (2, 128000, 64, 2.0 ** -10, 6, 4)])
def test_fp16_rows_of_any_weight(T, V, H, alpha, shift, decades):
    """Each row of dX, and each row of dW, is as exact as its own terms, however
    far apart the rows' weights and however small P (alpha 2^-10: logits that
    hardly differ, P = 1 / V; W off centre, so that its sum over the vocabulary
    counts).

    Logits are exact.  exp(l - lse) is off by at most ds = (60 + V / 8192) *
    2^-22 relative: 17 + V / 8192 and |lse| + 1 for the lse, |l - lse| / 2 + 3 for the
    exponential, |lse| and |l - lse| below 26 where it counts.  P times a power
    of two times dloss is rounded to FP16: u relative to the term or 2^-34 of its
    row's |dloss| in dX, 2^-39 of max|dloss| in dW.  These roundings are
    independent or, for equal terms, equal; the bound allows both.  A sum of n
    products in FP32: the matrix instruction adds 32 at a time, n / 32 + 8 sums in
    sequence, each off by 2^-23 of the sum of absolute terms.  The result is
    rounded to FP16."""
    torch = torch_cuda()
    X, W, t, d = spread(torch, T, V, H, shift, decades, 3)
    _, lse = lib.sgemm_xent(X, W, t, alpha=alpha)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d, alpha=alpha)
    _, _, rX, rW, aX, aW = xent_ref(torch, X, W, t, alpha, -100, d)
    un, ds = u(torch.float16, torch), (60 + V / 8192) * 2.0 ** -22
    own = (alpha * d.double())[:, None] * W.double().abs().sum(0)
    most = alpha * d.double().max() * X.double().abs().sum(0)
    assert_within(torch, dX, rX, (un + ds + (V / 32 + 8) * 2.0 ** -23) * aX + 2.0 ** -34 * own + 1.01 * un * rX.abs() + 2.0 ** -25, "dX")
    assert_within(torch, dW, rW, (un + ds + (T / 32 + 8) * 2.0 ** -23) * aW + 2.0 ** -39 * most + 1.01 * un * rW.abs() + 2.0 ** -25, "dW")


def test_fp16_rescaled_rows_do_not_change_with_what_is_asked_for():
    """dW is the same bits with and without dX, a captured graph replays them,
    and so does a vocabulary in pieces."""
    torch = torch_cuda()
    X, W, t, d = spread(torch, 300, 3001, 64, 0, 8, 5)
    _, lse = lib.sgemm_xent(X, W, t, alpha=0.125)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d, alpha=0.125)
    assert torch.equal(lib.sgemm_xent_grad(X, W, t, lse, d, alpha=0.125, need_dx=False)[1], dW)
    assert torch.equal(lib.sgemm_xent_grad(X, W, t, lse, d, alpha=0.125, need_dw=False)[0], dX)

    def run():
        return lib.sgemm_xent_grad(X, W, t, lse, d, alpha=0.125)

    def see(outs, i):
        for a, b in zip(outs, run()):
            assert torch.equal(a, b), f"replay {i}"
    replays(torch, run, lambda o: o, lambda i: d.copy_(spread(torch, 300, 3001, 64, 0, 3 * i, 7 + i)[3]), see)


def test_fp16_many_rows_in_pieces():
    torch = torch_cuda()
    X, W, t, d = problem(torch, 70000, 2501, 40, torch.float16, 0.25)
    d *= torch.logspace(0, -7, 70000, device="cuda")
    check(torch, X, W, t, d)
    _, lse = lib.sgemm_xent(X, W, t)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d * 2.0 ** 12)
    far = torch.arange(60000, 60100, device="cuda")                 # rows a millionth of the largest, on their own
    alone, _ = lib.sgemm_xent_grad(X[far], W, t[far], lse[far], d[far] * 2.0 ** 12)
    live = t[far] != -100
    # two results, each off by u for its own rounding and about u for its terms', which are independent
    err = (dX[far].double() - alone.double()).norm(dim=1) / alone.double().norm(dim=1)
    assert live.any() and (err[live] <= 4 * u(torch.float16, torch)).all()
    assert (dX[far][~live] == 0).all()


def test_fp16_infinite_weight_of_one_row():
    """dX of the other rows is what it is without that row (each of the two off
    by u for its own rounding and about u for its terms')."""
    torch = torch_cuda()
    X, W, t, _ = problem(torch, 40, 300, 64, torch.float16)
    d = torch.logspace(-3, 4, 40, device="cuda")
    _, lse = lib.sgemm_xent(X, W, t)
    want, _ = lib.sgemm_xent_grad(X, W, t, lse, d)
    d[7] = float("inf")
    dX, _ = lib.sgemm_xent_grad(X, W, t, lse, d)
    keep = torch.arange(40, device="cuda") != 7
    err = (dX[keep].double() - want[keep].double()).norm(dim=1) / want[keep].double().norm(dim=1)
    assert (err <= 4 * u(torch.float16, torch)).all() and not dX[7].isfinite().all()

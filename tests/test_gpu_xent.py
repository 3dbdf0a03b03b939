"""sgemm_xent and sgemm_xent_grad against the 64-bit formula.

Tolerances.  Logits: K products summed in FP32, off by at most
dl = K * 2^-23 * sum |x w| (times |alpha|); 0 for integer inputs.  lse: each
exp(l - top) is off by at most (2 + |l - top|) * 2^-22 relative (the rounded
argument l - top times log2(e), and the instruction's step), which weighted by
exp(l - top) is at most 3 * 2^-22 of the sum per term; the sum adds at most
40 + V / 2048 + 16 partial sums in sequence, each off by 2^-24 relative; so lse is off by at
most ds = (3 + 14 + V / 8192) * 2^-22 + dl, plus 2^-22 * (|lse| + 1) for the
logarithm and the last roundings, and the loss by that plus dl.
Gradients: P * dloss / max is rounded to the inputs' type once (u per term, or
half of the smallest fp16 step 2^-25 * max|dloss|), P itself is off by exp of
the errors of l and lse, and the sums run in FP32:
  |err| <= (u + 2 (dl + ds) + n * 2^-23) * sum |terms| + 2^-25 * max|dloss| * sum |other operand|
plus the final rounding u * |gradient|, subnormal step 2^-25.  Where exp(l - lse)
lies below the smallest normal number 2^-126 it may count as 0, so each term is
off by up to 2^-126 * max|dloss| * |other operand| besides, and so may a result
below 2^-126 (rows of exact logits far apart have such terms alone).
"""
import pytest

import fp32_sgemm_tuning_amd as lib
from fp32_sgemm_tuning_amd import capi
from gpu_util import torch_cuda
from products_util import assert_equal, assert_within, ints, normal, padded, replays, u, xent_ref

pytestmark = pytest.mark.gpu

IGNORE = -100


def problem(torch, T, V, H, dtype, ignored=0.0, seed=0, scale=None):
    X, W = normal(torch, (T, H), dtype, seed + 1), normal(torch, (V, H), dtype, seed + 2, scale or 3 * max(H, 1) ** -0.5)
    g = torch.Generator().manual_seed(seed + 3)
    target = torch.randint(0, V, (T,), generator=g)
    target[torch.rand(T, generator=g) < ignored] = IGNORE
    dloss = torch.rand(T, generator=g) + 0.25
    return X, W, target.cuda(), dloss.cuda()


def check(torch, X, W, target, dloss, alpha=1.0, ignore=IGNORE, outs=None, what=""):
    T, H = X.shape
    V = W.shape[0]
    loss, lse = lib.sgemm_xent(X, W, target, alpha=alpha, ignore_index=ignore) if outs is None else outs[:2]
    dX, dW = lib.sgemm_xent_grad(X, W, target, lse, dloss, alpha=alpha, ignore_index=ignore) if outs is None else outs[2:]
    rloss, rlse, rX, rW, aX, aW = xent_ref(torch, X, W, target, alpha, ignore, dloss)
    live = target != ignore
    Xl = torch.where(live[:, None], X, torch.zeros_like(X))
    dl = abs(alpha) * H * 2.0 ** -23 * (Xl.double().abs() @ W.double().abs().amax(0)[:, None]).amax()
    ds = (17 + V / 8192) * 2.0 ** -22 + dl
    tol = ds + dl + 2.0 ** -22 * (2 * rlse.abs() + rloss.abs() + 1)
    assert_within(torch, lse, rlse, torch.where(live, tol, 0.0), f"lse {what}")
    assert_within(torch, loss, rloss, torch.where(live, tol, 0.0), f"loss {what}")
    un, top = u(X.dtype, torch), dloss.double().abs().max() * abs(alpha)
    step = 2.0 ** -25 if X.dtype == torch.float16 else 2.0 ** -126
    Wsum, Xsum = W.double().abs().sum(0), Xl.double().abs().sum(0)
    assert_within(torch, dX, rX, (un + 2 * (dl + ds) + V * 2.0 ** -23) * aX + un * rX.abs() * 1.01
                  + torch.where(live, step * top, 0.0)[:, None] * Wsum + step, f"dX {what}")
    assert_within(torch, dW, rW, (un + 2 * (dl + ds) + T * 2.0 ** -23) * aW + un * rW.abs() * 1.01 + step * top * Xsum
                  + step, f"dW {what}")
    assert (dX[~live] == 0).all() and (loss[~live] == 0).all() and (lse[~live] == 0).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("T,V,H,ignored", [
    (1, 1000, 64, 0.0), (1, 1, 8, 0.0), (3, 7, 72, 0.0), (17, 129, 64, 0.3), (33, 1000, 1, 0.0), (64, 1023, 37, 0.5),
    (130, 511, 200, 0.9), (257, 1537, 264, 0.1), (500, 300, 131, 0.0), (1000, 5003, 128, 0.4), (2048, 8192, 64, 0.0),
    (700, 33001, 96, 0.2)])
def test_against_formula(T, V, H, ignored, dtype):
    torch = torch_cuda()
    check(torch, *problem(torch, T, V, H, getattr(torch, dtype), ignored))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_vocabulary_in_pieces(dtype):
    """So many rows that the backward takes the vocabulary in two pieces."""
    torch = torch_cuda()
    T, V, H = 70000, 2501, 40
    pieces = capi.sgemm_lowp_xent_workspace(T, V, H, 0x1000, H, 0x1000, H, 1)
    assert pieces < T * V * 2 + 3 * T * H * 4
    check(torch, *problem(torch, T, V, H, getattr(torch, dtype), 0.25))


@pytest.mark.parametrize("T", [16384, 16385, 40001])
def test_many_rows(T):
    """Above 16384 rows they are counted by segments first."""
    torch = torch_cuda()
    check(torch, *problem(torch, T, 300, 16, torch.bfloat16, 0.5))


@pytest.mark.parametrize("alpha", [0.25, -1.0, 0.0])
def test_scaled_logits(alpha):
    torch = torch_cuda()
    check(torch, *problem(torch, 40, 300, 64, torch.bfloat16, 0.2), alpha=alpha)


def test_integer_logits():
    """Exact logits far apart: one term rules each sum, and rows of equal
    logits give log(V)."""
    torch = torch_cuda()
    X, W = ints(torch, (50, 64), -4, 4, torch.bfloat16, 1), ints(torch, (400, 64), -4, 4, torch.bfloat16, 2)
    X[7] = 0
    t = (torch.arange(50, device="cuda") * 7) % 400
    check(torch, X, W, t, torch.full((50,), 0.5, device="cuda"))
    loss, lse = lib.sgemm_xent(X, W, t)
    assert abs(lse[7].item() - 5.991464547107982) < 1e-5 and abs(loss[7].item() - 5.991464547107982) < 1e-5


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), -3e38])
@pytest.mark.parametrize("T,H", [(90, 64), (90, 61), (20, 64), (20, 61)])
def test_ignored_rows_may_hold_anything(T, H, fill):
    torch = torch_cuda()
    X, W, t, d = problem(torch, T, 260, H, torch.bfloat16, 0.4)
    ignored = t == IGNORE
    X[ignored] = fill
    d[ignored] = float("nan")
    loss, lse = lib.sgemm_xent(X, W, t)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d)
    check(torch, torch.where(ignored[:, None], torch.zeros_like(X), X), W, t, torch.where(ignored, 0.0, d),
          outs=(loss, lse, dX, dW))


def test_all_rows_ignored():
    torch = torch_cuda()
    X, W, t, d = problem(torch, 20, 260, 64, torch.float16)
    t.fill_(5)
    X.fill_(float("nan"))
    loss, lse = lib.sgemm_xent(X, W, t, ignore_index=5)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d, ignore_index=5)
    for o in (loss, lse, dX, dW):
        assert (o == 0).all()


def test_target_outside_the_vocabulary():
    """NaN for that row (and for dW), the other rows unharmed; a target that
    only looks small in 32 bits is outside too."""
    torch = torch_cuda()
    X, W, t, d = problem(torch, 30, 100, 64, torch.bfloat16)
    t[3], t[4], t[5] = 100, -1, 2 ** 32 + 1
    loss, lse = lib.sgemm_xent(X, W, t)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d)
    bad = torch.zeros(30, dtype=torch.bool, device="cuda")
    bad[3:6] = True
    assert torch.equal(loss.isnan(), bad) and not lse.isnan().any()
    assert dX[bad].isnan().all() and not dX[~bad].isnan().any() and dW.isnan().all()


def test_infinite_and_nan_logits():
    """-inf logits have no part in the sum, as in the formula; a NaN makes its
    own row NaN only."""
    torch = torch_cuda()
    X, W, t, _ = problem(torch, 12, 300, 8, torch.bfloat16)
    X = X.abs() + 0.1
    W[10] = -float("inf")
    t[:] = 20
    X[5, 0] = float("nan")
    loss, lse = lib.sgemm_xent(X, W, t)
    keep = torch.arange(12, device="cuda") != 5
    W2 = torch.cat([W[:10], W[11:]])
    rloss, rlse = xent_ref(torch, X[keep], W2, t[keep] - 1)
    assert loss[5].isnan() and lse[5].isnan()
    tol = 40 * 2.0 ** -22 * (rlse.abs() + 1)
    assert_within(torch, lse[keep], rlse, tol)
    assert_within(torch, loss[keep], rloss, tol + 20 * 2.0 ** -22)


def test_dloss_forms():
    torch = torch_cuda()
    X, W, t, _ = problem(torch, 45, 300, 64, torch.float16, 0.2)
    _, lse = lib.sgemm_xent(X, W, t)
    one = lib.sgemm_xent_grad(X, W, t, lse, torch.full((45,), 0.125, device="cuda"))
    for d in (torch.tensor(0.125, device="cuda"), torch.tensor([0.125], device="cuda"),
              torch.full((90,), 0.125, device="cuda")[::2], torch.tensor(0.125, device="cuda").expand(45)):
        for a, b in zip(one, lib.sgemm_xent_grad(X, W, t, lse, d)):
            assert torch.equal(a, b)
    # a loss scale does not cost precision: powers of two scale the result exactly
    up = lib.sgemm_xent_grad(X, W, t, lse, torch.tensor(0.125 * 2.0 ** -40, device="cuda"))
    down = lib.sgemm_xent_grad(X.bfloat16(), W.bfloat16(), t, lse, torch.tensor(0.125 * 2.0 ** -40, device="cuda"))
    same = lib.sgemm_xent_grad(X.bfloat16(), W.bfloat16(), t, lse, torch.tensor(0.125, device="cuda"))
    assert (up[0] == 0).all()                        # fp16 has no such values
    assert torch.equal(down[0].float() * 2.0 ** 40, same[0].float())
    zero = lib.sgemm_xent_grad(X, W, t, lse, torch.zeros(45, device="cuda"))
    assert (zero[0] == 0).all() and (zero[1] == 0).all()
    inf = torch.full((45,), 0.5, device="cuda")
    live = (t != IGNORE).nonzero()[:, 0]
    inf[live[0]] = float("inf")
    dX, _ = lib.sgemm_xent_grad(X, W, t, lse, inf)
    assert not dX[live[1:]].isnan().any()


def test_only_one_gradient():
    torch = torch_cuda()
    X, W, t, d = problem(torch, 45, 300, 64, torch.bfloat16, 0.2)
    _, lse = lib.sgemm_xent(X, W, t)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d)
    a, none = lib.sgemm_xent_grad(X, W, t, lse, d, need_dw=False)
    assert none is None and torch.equal(a, dX)
    none, b = lib.sgemm_xent_grad(X, W, t, lse, d, need_dx=False)
    assert none is None and torch.equal(b, dW)
    assert lib.sgemm_xent_grad(X, W, t, lse, d, need_dx=False, need_dw=False) == (None, None)


def test_no_rows():
    torch = torch_cuda()
    X, W = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), normal(torch, (50, 64), torch.bfloat16, 1)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = lib.sgemm_xent(X, W, t)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, torch.empty(0, device="cuda"))
    assert loss.shape == lse.shape == (0,) and dX.shape == (0, 64) and (dW == 0).all()


@pytest.mark.parametrize("pad,base", [(8, 0), (8, 8), (3, 0), (0, 1)])
def test_strides(pad, base):
    torch = torch_cuda()
    X, W, t, d = problem(torch, 200, 515, 72, torch.bfloat16, 0.3)
    check(torch, padded(torch, X, pad, base), padded(torch, W, pad, base), t, d)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss along a direction: their error is
    h^2 / 6 times the third derivative, below 1e-7 here; the product of the
    direction with the gradient is off by at most the gradient's own bound."""
    torch = torch_cuda()
    X, W, t, d = problem(torch, 24, 90, 32, torch.bfloat16, 0.2)
    _, lse = lib.sgemm_xent(X, W, t)
    dX, dW = lib.sgemm_xent_grad(X, W, t, lse, d)
    vX, vW = normal(torch, X.shape, torch.float64, 8), normal(torch, W.shape, torch.float64, 9)
    h = 1e-4

    def value(x, w):
        l = x @ w.T.contiguous()
        rows = (t != IGNORE).nonzero()[:, 0]
        return (d.double()[rows] * (torch.logsumexp(l[rows], 1) - l[rows, t[rows]])).sum()
    x, w = X.double(), W.double()
    aX, aW = xent_ref(torch, X, W, t, 1.0, IGNORE, d)[4:]
    for grad, v, big, plus, minus in ((dX, vX, aX, (x + h * vX, w), (x - h * vX, w)),
                                      (dW, vW, aW, (x, w + h * vW), (x, w - h * vW))):
        slope = (value(*plus) - value(*minus)) / (2 * h)
        tol = (2 ** -7 + 2 ** -10) * (big * v.abs()).sum() + 1e-5
        assert abs((grad.double() * v).sum() - slope) <= tol
        # an estimate of the true error, far tighter than the bound: rounding errors are independent
        assert abs((grad.double() * v).sum() - slope) <= 8 * 2 ** -8 * ((big * v) ** 2).sum().sqrt()


def test_captured_with_new_inputs():
    torch = torch_cuda()
    X, W, t, d = problem(torch, 150, 1100, 72, torch.float16, 0.3)
    news = [problem(torch, 150, 1100, 72, torch.float16, 0.1 * i, seed=10 * i) for i in range(3)]

    def run():
        loss, lse = lib.sgemm_xent(X, W, t)
        return (loss, lse, *lib.sgemm_xent_grad(X, W, t, lse, d))

    def refresh(i):
        for a, b in zip((X, W, t, d), news[i]):
            a.copy_(b)

    def see(outs, i):
        check(torch, X, W, t, d, outs=outs, what=f"replay {i}")
        for a, b in zip(outs, run()):
            assert torch.equal(a, b)
    replays(torch, run, lambda o: o, refresh, see)


def test_two_streams_at_once():
    torch = torch_cuda()
    cases = [problem(torch, 300 + i, 2000, 64, torch.bfloat16, 0.2, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for c, s in zip(cases, streams):
            loss, lse = lib.sgemm_xent(*c[:3], stream=s)
            outs.append((c, (loss, lse, *lib.sgemm_xent_grad(*c[:3], lse, c[3], stream=s))))
    torch.cuda.synchronize()
    for c, o in outs:
        check(torch, *c, outs=o)


def test_race_check_build(monkeypatch):
    torch = torch_cuda()
    monkeypatch.setattr(capi, "_lib", capi.open_library(capi.POISON_LIB_PATH))
    for T, V, H in ((20, 700, 200), (300, 1500, 264), (2100, 9000, 264)):
        check(torch, *problem(torch, T, V, H, torch.bfloat16, 0.1))


def test_refusals():
    torch = torch_cuda()
    X, W, t, d = problem(torch, 6, 10, 8, torch.bfloat16)
    loss, lse = lib.sgemm_xent(X, W, t)
    for bad in (dict(X=X.float()), dict(W=W.half()), dict(target=t.int())):
        with pytest.raises(TypeError):
            lib.sgemm_xent(**{**dict(X=X, W=W, target=t), **bad})
    for bad in (dict(W=W[:, :4]), dict(target=t[:5]), dict(W=W[:0]), dict(X=X[None]), dict(X=X.cpu()),
                dict(target=t.cpu()), dict(target=t[:, None]), dict(W=W.T)):
        with pytest.raises(ValueError):
            lib.sgemm_xent(**{**dict(X=X, W=W, target=t), **bad})
    for bad in (dict(dloss=d.double()), dict(lse=lse.double())):
        with pytest.raises(TypeError):
            lib.sgemm_xent_grad(**{**dict(X=X, W=W, target=t, lse=lse, dloss=d), **bad})
    for bad in (dict(dloss=d[:5]), dict(lse=lse[:5]), dict(dloss=d[:, None]), dict(lse=lse.cpu())):
        with pytest.raises(ValueError):
            lib.sgemm_xent_grad(**{**dict(X=X, W=W, target=t, lse=lse, dloss=d), **bad})

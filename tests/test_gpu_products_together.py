"""The operators as a model uses them together: a training step of an expert
layer under an output layer with its loss, then one token's logits from the
same output weight in 4 bits."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import normal

pytestmark = pytest.mark.gpu


def _plain(torch, x, experts, out, off, target, valid):
    """Loss and gradients of the same step in 64 bits by automatic differentiation."""
    x, experts, out = (t.double().requires_grad_() for t in (x, experts, out))
    h = torch.cat([x[a:b] @ experts[g] for g, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    logits = h @ out.T
    loss = torch.logsumexp(logits, 1) - logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    loss = (loss * valid).sum() / valid.sum()
    loss.backward()
    return loss.detach(), x.grad, experts.grad, out.grad


def test_training_step_then_token():
    torch = torch_cuda()
    T, G, K, H, V = 333, 4, 72, 136, 1003
    e = torch.bfloat16
    off = [0, 100, 100, 101, 333]
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, experts = normal(torch, (T, K), e, 1), normal(torch, (G, K, H), e, 2, K ** -0.5)
    out = normal(torch, (V, H), e, 3, H ** -0.5)
    target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(4)).cuda()
    target[::5] = -100
    valid = target >= 0
    h = lib.sgemm_grouped(x, experts, dev, out_dtype=e)
    loss, lse = lib.sgemm_xent(h, out, target)
    dh, dout = lib.sgemm_xent_grad(h, out, target, lse, 1.0 / valid.sum().float())
    dx = lib.sgemm_grouped(dh, experts, dev, trans_b=True)
    dexperts = lib.sgemm_grouped_wgrad(x, dh, dev)
    rloss, rx, rexperts, rout = _plain(torch, x, experts, out, off, target, valid)
    # h is rounded to 16 bits (2^-8 at most, about 2^-9 / sqrt(3) * 2 in the mean), dh twice: four such
    # roundings of independent terms stay below 2^-7 of the norm
    assert abs(loss.double().sum() / valid.sum() - rloss) < 2 ** -7
    for got, ref in ((dx, rx), (dexperts, rexperts), (dout, rout)):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 2 ** -7
    W = lib.sgemm_w4_quantize(out, group=32, zeros=True)
    token = h[7:8]
    logits = lib.sgemm_w4(token, W)
    values = lib.sgemm_w4_dequantize(W).double()
    ref = token.double() @ values.T.contiguous()
    # the product takes the weights unrounded, the values were rounded once to bf16
    assert ((logits.double() - ref).abs() <= 2 ** -7 * (token.double().abs() @ values.abs().T.contiguous())).all()
    assert ((logits.double() - ref).norm() / ref.norm()).item() < 2 ** -8


def test_weights_past_32_bits():
    """Weights of more than 2^32 bytes (the last rows of each lie behind)."""
    torch = torch_cuda()
    e = torch.bfloat16
    # (products of -1, 0 and 1: sums are exact)
    B = torch.randint(-1, 2, (3, 32768, 32768), device="cuda", dtype=torch.int8).to(e)
    A = torch.randint(-1, 2, (70, 32768), device="cuda", dtype=torch.int8).to(e)
    dev = torch.tensor([0, 20, 30, 70], dtype=torch.int32, device="cuda")
    C = lib.sgemm_grouped(A, B, dev)
    assert torch.equal(C[30:, -300:].double(), A[30:].double() @ B[2][:, -300:].double().contiguous())
    C = lib.sgemm_grouped(A, B, dev, trans_b=True)
    assert torch.equal(C[30:, -300:].double(), A[30:].double() @ B[2][-300:].double().T.contiguous())
    del B, C
    D = torch.randint(-1, 2, (70, 32768), device="cuda", dtype=torch.int8).to(e)
    G = lib.sgemm_grouped_wgrad(A, D, dev, out_dtype=e)
    assert torch.equal(G[2][-300:].double(), A[30:, -300:].double().T.contiguous() @ D[30:].double())
    del G
    W = torch.randint(-1, 2, (600001, 4096), device="cuda", dtype=torch.int8).to(e)
    X = torch.randint(-1, 2, (40, 4096), device="cuda", dtype=torch.int8).to(e)
    target = torch.arange(600001 - 40, 600001, device="cuda")
    loss, lse = lib.sgemm_xent(X, W, target, alpha=2.0 ** -6)
    logits = torch.cat([2.0 ** -6 * (X.double() @ w.double().T.contiguous()) for w in W.split(50000)], 1)
    ref = torch.logsumexp(logits, 1)
    # exact logits: lse is off by (17 + V / 8192) * 2^-22 at most for the exponentials and the sum, and the logarithm
    tol = (17 + 600001 / 8192) * 2 ** -22 + 2 ** -21 * (ref.abs() + 1)
    assert ((lse.double() - ref).abs() <= tol).all()
    rows = torch.arange(40, device="cuda")
    assert ((loss.double() - (ref - logits[rows, target])).abs() <= 2 * tol).all()
    _, dW = lib.sgemm_xent_grad(X, W, target, lse, torch.ones(40, device="cuda"), alpha=2.0 ** -6, need_dx=False)
    P = torch.exp(logits[:, -100:] - ref[:, None])
    P[rows, 60 + rows] -= 1
    want = 2.0 ** -6 * (P.T.contiguous() @ X.double())
    big = 2.0 ** -6 * (P.abs().T.contiguous() @ X.double().abs())
    assert ((dW[-100:].double() - want).abs() <= (2 ** -8 + 2 ** -12) * big + 2 ** -8 * want.abs()).all()
    del W, dW, logits
    packed = torch.randint(0, 256, (300000, 16384), dtype=torch.uint8, device="cuda")
    scales = torch.ones(300000, 256, dtype=e, device="cuda")
    for M in (1, 100):
        x = torch.randint(-1, 2, (M, 32768), device="cuda", dtype=torch.int8).to(e)
        whole = lib.sgemm_w4(x, lib.W4Weight(packed, scales, None, 32768, 128))
        last = lib.W4Weight(packed[-70:].clone(), scales[-70:].clone(), None, 32768, 128)
        assert torch.equal(whole[:, -70:], lib.sgemm_w4(x, last))
        values = lib.sgemm_w4_dequantize(last).double()        # exact in bf16 here
        assert torch.equal(whole[:, -70:].double(), x.double() @ values.T.contiguous())
    tail = lib.sgemm_w4_dequantize(lib.W4Weight(packed, scales, None, 32768, 128))[-70:]
    assert torch.equal(tail.double(), values)

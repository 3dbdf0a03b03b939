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

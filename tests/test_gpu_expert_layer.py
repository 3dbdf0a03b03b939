"""Routing and products as an expert layer uses them together: a training step
in 16 bits, and a serving step in 8-bit integers."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import normal

pytestmark = pytest.mark.gpu


def _layer(torch, x, experts, weights, up, down):
    """sum over picks of weights * (silu(x @ up[e]) @ down[e]) in 64 bits, picks of no expert left out."""
    out = torch.zeros_like(x)
    for g in range(up.shape[0]):
        for j in range(experts.shape[1]):
            t = (experts[:, j] == g).nonzero()[:, 0]
            if len(t):
                out = out.index_add(0, t, weights[t, j, None] * (torch.nn.functional.silu(x[t] @ up[g]) @ down[g]))
    return out


def test_training_step():
    torch = torch_cuda()
    T, picks, G, H, F = 217, 3, 6, 72, 136
    e = torch.bfloat16
    x, D = normal(torch, (T, H), e, 1), normal(torch, (T, H), e, 4)
    up, down = normal(torch, (G, H, F), e, 2, H ** -0.5), normal(torch, (G, F, H), e, 3, F ** -0.5)
    gen = torch.Generator().manual_seed(5)
    experts = torch.randn(T, G, generator=gen).topk(picks, 1).indices.cuda()
    experts[::9] = -1
    weights = torch.softmax(torch.randn(T, picks, generator=gen), 1).cuda()

    rows, order = lib.sgemm_grouped_sort(x, experts, G)
    a = torch.zeros(T * picks, F, dtype=e, device="cuda")
    lib.sgemm_grouped(rows, up, order.offsets, a)
    h = torch.nn.functional.silu(a.float()).to(e)
    y = torch.zeros(T * picks, H, dtype=e, device="cuda")
    lib.sgemm_grouped(h, down, order.offsets, y)
    out = lib.sgemm_grouped_combine(y, order, weights)
    dy, dweights = lib.sgemm_grouped_combine_grad(D, y, order, weights)
    ddown = lib.sgemm_grouped_wgrad(h, dy, order.offsets)
    dh = torch.zeros(T * picks, F, device="cuda")
    lib.sgemm_grouped(dy, down, order.offsets, dh, trans_b=True)
    s = torch.sigmoid(a.float())
    da = (dh * s * (1 + a.float() * (1 - s))).to(e)
    dup = lib.sgemm_grouped_wgrad(rows, da, order.offsets)
    drows = torch.zeros(T * picks, H, dtype=e, device="cuda")
    lib.sgemm_grouped(da, up, order.offsets, drows, trans_b=True)
    dx = lib.sgemm_grouped_combine(drows, order)

    leaves = [v.double().requires_grad_() for v in (x, weights, up, down)]
    ref = _layer(torch, leaves[0], experts, leaves[1], *leaves[2:])
    (ref * D.double()).sum().backward()
    # up to seven roundings to 16 bits on the way to a result (each 2^-8 at most of its value, about
    # 2^-9 / sqrt(3) of the norm): below 2^-6 of the norm
    for got, want in ((out, ref.detach()), (dx, leaves[0].grad), (dweights, leaves[1].grad), (dup, leaves[2].grad), (ddown, leaves[3].grad)):
        assert ((got.double() - want).norm() / want.norm()).item() < 2 ** -6
    assert (out[::9] == 0).all() and (dx[::9] == 0).all() and (dweights[::9] == 0).all()


@pytest.mark.parametrize("T", [1, 4, 300])
def test_serving_step_in_8_bits(T):
    torch = torch_cuda()
    picks, G, H, F = 2, 8, 200, 328
    x = normal(torch, (T, H), torch.bfloat16, 1)
    up = lib.sgemm_i8_quantize(normal(torch, (G, F, H), torch.bfloat16, 2, H ** -0.5))
    down = lib.sgemm_i8_quantize(normal(torch, (G, H, F), torch.bfloat16, 3, F ** -0.5))
    gen = torch.Generator().manual_seed(5)
    experts = torch.randn(T, G, generator=gen).topk(picks, 1).indices.int().cuda()
    weights = torch.softmax(torch.randn(T, picks, generator=gen), 1).cuda()
    q = lib.sgemm_i8_quantize(x)
    rows, order = lib.sgemm_grouped_sort(q, experts, G)
    h = torch.nn.functional.silu(lib.sgemm_i8_grouped(rows, up, order.offsets))
    hq = lib.sgemm_i8_quantize(h)
    y = lib.sgemm_i8_grouped(hq, down, order.offsets, out_dtype=torch.bfloat16)
    out = lib.sgemm_grouped_combine(y, order, weights)
    # the same with the values that the 8 bits stand for: the products are exact but for roundings to FP32
    # (and of y and out to bf16), the hidden values as quantised
    U, V, X = (lib.sgemm_i8_dequantize(m).double() for m in (up, down, q))
    Hd = lib.sgemm_i8_dequantize(hq).double()
    for t in range(T):
        want = torch.zeros(H, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for j in range(picks):
            g, r = int(experts[t, j]), int(order.position[t, j])
            pre = U[g] @ X[t]
            near = torch.nn.functional.silu(pre)
            # h before quantisation, in FP32; its step is rounded to at most half a scale
            assert ((h[r].double() - near).abs() <= 2 ** -18 * (1 + near.abs())).all()
            assert ((Hd[r] - h[r].double()).abs() <= hq.scales[r].double() * (0.5 + 2 ** -16)).all()
            term = weights[t, j].double() * (V[g] @ Hd[r])
            want, size = want + term, size + term.abs()
        # y rounded to bf16 (2^-9 of each term's size at most 2^-8), the sum once more
        assert ((out[t].double() - want).abs() <= 2 ** -8 * size + 2 ** -8 * want.abs() + 2 ** -20 * size).all()

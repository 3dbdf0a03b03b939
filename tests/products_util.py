"""Plain 64-bit forms of the grouped products, the output layer with its loss
and the 4-bit weights, and the rounding bounds the tests hold results to.

Bounds.  u(t) = finfo(t).eps / 2 is the largest relative error of one rounding
to t.  A sum of n products of exactly represented 16-bit values in FP32 is off
by at most n * 2^-23 * sum |a b| (n additions, each off by one step where the
matrix instruction truncates).  Integer-valued inputs with sums below 2^24 are
summed exactly, so there a result equals its 64-bit value rounded once.
"""
import numpy as np


def u(dtype, torch):
    return torch.finfo(dtype).eps / 2


def ints(torch, shape, lo, hi, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g).to(dtype).cuda()


def normal(torch, shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def padded(torch, x, pad, offset=0, fill=float("nan")):
    """x as a view with `pad` more elements per row, `offset` elements into
    its allocation, everything outside it NaN."""
    rows, cols = x.shape[-2:]
    lead = x.numel() // max(rows * cols, 1)
    ld = cols + pad
    buf = torch.full((offset + max(lead, 1) * rows * ld + 8,), fill, dtype=x.dtype, device=x.device)
    view = buf[offset:offset + lead * rows * ld].view(*x.shape[:-2], rows, ld)[..., :cols]
    view.copy_(x)
    return view


def grouped_ref(torch, A, B, offsets, trans_b):
    """(C, rows that belong to a group) in 64 bits."""
    A, B = A.double(), B.double()
    N = B.shape[1] if trans_b else B.shape[2]
    C = torch.zeros(A.shape[0], N, dtype=torch.float64, device=A.device)
    live = torch.zeros(A.shape[0], dtype=torch.bool, device=A.device)
    for g, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        W = B[g].T if trans_b else B[g]
        C[a:b] = A[a:b] @ W.contiguous()
        live[a:b] = True
    return C, live


def wgrad_ref(torch, A, D, offsets):
    return torch.stack([A[a:b].double().T.contiguous() @ D[a:b].double()
                        for a, b in zip(offsets[:-1], offsets[1:])])


def xent_ref(torch, X, W, target, alpha=1.0, ignore=-100, dloss=None):
    """loss, lse and (with dloss) dX, dW, and the sums of absolute terms of
    dX and dW, in 64 bits; ignored rows take no part."""
    rows = (target != ignore).nonzero()[:, 0]
    X, W = X.double(), W.double()
    loss = torch.zeros(len(target), dtype=torch.float64, device=X.device)
    lse = torch.zeros_like(loss)
    dX, dW, aX, aW = torch.zeros_like(X), torch.zeros_like(W), torch.zeros_like(X), torch.zeros_like(W)
    for r in rows.split(4096):
        l = alpha * (X[r] @ W.T.contiguous())
        lse[r] = torch.logsumexp(l, 1)
        i = torch.arange(len(r), device=X.device)
        loss[r] = lse[r] - l[i, target[r]]
        if dloss is not None:
            P = torch.exp(l - lse[r][:, None])
            P[i, target[r]] -= 1
            P *= alpha * dloss.double().expand(len(target))[r][:, None]
            dX[r], dW = P @ W, dW + P.T.contiguous() @ X[r]
            aX[r], aW = P.abs() @ W.abs(), aW + P.abs().T.contiguous() @ X[r].abs()
    return (loss, lse) if dloss is None else (loss, lse, dX, dW, aX, aW)


def w4_values(torch, W):
    """(q - z) and s of a W4Weight as 64-bit [N,K] arrays, read with numpy
    from the documented layout."""
    N, K, group = W.packed.shape[0], W.K, W.group
    words = W.packed.cpu().numpy().view("<u4").astype(np.int64)
    k = np.arange(K)
    inside = k % 128
    word = k // 128 * 16 + 4 * (inside % 32 // 8) + inside // 32
    e = k % 8
    q = (words[:, word] >> (4 * (e // 2) + 16 * (e % 2))) & 15
    z = 8 if W.zeros is None else W.zeros.cpu().numpy().astype(np.int64)[:, k // group]
    s = W.scales.double().cpu().numpy()[:, k // group]
    return torch.from_numpy((q - z).astype(np.float64)).reshape(N, K).cuda(), torch.from_numpy(s).reshape(N, K).cuda()


def assert_within(torch, got, ref, tol, what=""):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values out of tolerance, first at "
                           f"{bad.nonzero()[0].tolist()}: got {got[bad][0].item()!r} want {ref[bad][0].item()!r}")


def assert_equal(torch, got, ref64, what=""):
    """got equals the 64-bit values rounded once to its type."""
    want = ref64.to(got.dtype)
    bad = ~(got == want)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values differ, first at "
                           f"{bad.nonzero()[0].tolist()}: got {got[bad][0].item()!r} want {want[bad][0].item()!r}")


def replays(torch, run, outputs, refresh, check, times=3):
    """Captures run(), then replays it with new inputs, the program's own
    eager work and synchronisations in between; check() sees every replay."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i in range(times):
        refresh(i)
        for o in outputs(outs):
            o.zero_()
        torch.ones(1 << 18, device="cuda").cumsum(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(outs, i)

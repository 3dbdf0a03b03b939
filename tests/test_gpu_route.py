"""Tokens sorted by expert and back, with weights, and the gradients, against
plain forms in 64 bits.

Tolerances.  Places and copied rows are exact.  A sum of p products in FP32,
each of them rounded at most once and added with one rounding, is off by at most
2 p * 2^-24 * (1 + 2^-20) of the sum of the absolute terms, a dot product of H
terms by H + 1 roundings of them at most; then one rounding to the result's
type."""
import pytest

import fp32_sgemm_tuning_amd as lib
from gpu_util import torch_cuda
from products_util import assert_within, normal, padded, replays, u

pytestmark = pytest.mark.gpu

# (T, picks, groups): one launch, several, many groups; sizes around their borders
ORDERS = [(1, 1, 1), (1, 8, 256), (4, 2, 8), (7, 3, 5), (33, 1, 4), (64, 1, 64), (65, 1, 3), (100, 6, 60), (2048, 1, 16), (256, 8, 300),
          (2049, 1, 16), (4096, 1, 5), (512, 8, 64), (4097, 1, 16), (1366, 3, 4096), (1000, 7, 1), (3001, 6, 60), (5000, 2, 2047), (4000, 3, 2048), (16384, 8, 128), (40000, 4, 4096), (70001, 2, 7)]


def experts_of(torch, T, picks, groups, seed, dtype=None, drop=0.2):
    """Experts of uneven popularity, the same one twice in a token now and then; a share of none (values below 0 and above)."""
    g = torch.Generator().manual_seed(seed)
    e = (torch.rand(T, picks, generator=g) ** 2 * groups).long().clamp(max=max(groups - 1, 0))
    none = torch.rand(T, picks, generator=g) < drop
    e[none] = torch.tensor([-1, groups, -2 ** 31, 2 ** 31 - 1])[torch.randint(0, 4, (int(none.sum()),), generator=g)]
    return e.to(dtype or torch.int64).cuda()


def order_ref(torch, experts, groups):
    e = experts.cpu().long().reshape(-1)
    key = torch.where((e >= 0) & (e < groups), e, groups)
    source = torch.sort(key, stable=True).indices
    offsets = torch.tensor([int((key < g).sum()) for g in range(groups + 1)]) if groups < 100 else \
        torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(key, minlength=groups + 1)[:groups].cumsum(0)])
    position = torch.empty_like(source)
    position[source] = torch.arange(len(source))
    position[key == groups] = -1
    source[int(offsets[-1]):] = -1
    return offsets, position.view(experts.shape[0], -1), source


def check_order(torch, order, experts, groups):
    offsets, position, source = order_ref(torch, experts, groups)
    for got, want, name in zip(order, (offsets, position, source), ("offsets", "position", "source")):
        assert got.dtype == torch.int32 and torch.equal(got.cpu().long(), want), name
    return offsets, position, source


@pytest.mark.parametrize("T,picks,groups", ORDERS)
@pytest.mark.parametrize("wide", [False, True])
def test_order(T, picks, groups, wide):
    torch = torch_cuda()
    for drop in (0.0, 0.3, 1.0):
        e = experts_of(torch, T, picks, groups, T + picks, torch.int64 if wide else torch.int32, drop)
        rows, order = lib.sgemm_grouped_sort(None, e, groups)
        assert rows is None
        check_order(torch, order, e, groups)


@pytest.mark.parametrize("T,picks,groups", [(5, 2, 4), (3001, 3, 9)])
def test_experts_beyond_32_bits(T, picks, groups):
    """64-bit values whose low 32 bits would be an expert are none."""
    torch = torch_cuda()
    e = experts_of(torch, T, picks, groups, 1)
    e[::2] += 2 ** 32
    e[1::4] -= 2 ** 33
    check_order(torch, lib.sgemm_grouped_sort(None, e, groups)[1], e, groups)


def test_order_of_views_and_empty():
    torch = torch_cuda()
    e = experts_of(torch, 500, 9, 12, 3)
    for v in (e[:, :4], e[::3, 2:5], e[:, 0], e[:, 8]):
        check_order(torch, lib.sgemm_grouped_sort(None, v, 12)[1], v if v.dim() == 2 else v[:, None], 12)
    x = torch.zeros(0, 16, device="cuda")
    rows, order = lib.sgemm_grouped_sort(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 5)
    assert rows.shape == (0, 16) and order.offsets.tolist() == [0] * 6 and order.position.shape == (0, 2)
    assert lib.sgemm_grouped_combine(rows, order).shape == (0, 16)
    for T in (3, 3000):                         # no groups, no picks, no columns
        e = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
        rows, order = lib.sgemm_grouped_sort(torch.ones(T, 8, device="cuda"), e, 0)
        assert order.offsets.tolist() == [0] and (order.position == -1).all() and (order.source == -1).all() and (rows == 0).all()
        assert (lib.sgemm_grouped_combine(rows, order) == 0).all()
        rows, order = lib.sgemm_grouped_sort(torch.ones(T, 8, device="cuda"), e[:, :0], 2)
        assert rows.shape == (0, 8) and order.offsets.tolist() == [0, 0, 0]
        assert torch.equal(lib.sgemm_grouped_combine(rows, order), torch.zeros(T, 8, device="cuda"))
        rows, order = lib.sgemm_grouped_sort(torch.ones(T, 0, device="cuda"), e, 2)
        assert rows.shape == (2 * T, 0) and order.offsets.tolist() == [0, 2 * T, 2 * T]
        w = torch.ones(T, 2, device="cuda")
        dy, dw = lib.sgemm_grouped_combine_grad(torch.ones(T, 0, device="cuda"), rows, order, w)
        assert dy.shape == (2 * T, 0) and (dw == 0).all()


def test_no_assignments_and_no_rows():
    """Where there is no row to copy, X is not read."""
    torch = torch_cuda()
    offsets, rows = torch.full((4,), 7, dtype=torch.int32, device="cuda"), torch.full((16,), 3.0, device="cuda")
    st = lib.capi.sgemm_grouped_sort(lib.capi.SGEMM_DTYPE_F32, 5, 0, 3, 16, None, 16, None, None, 0, 4, offsets.data_ptr(), None, None,
                                     rows.data_ptr(), 16, None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == lib.capi.SGEMM_STATUS_OK
    assert offsets.tolist() == [0] * 4 and (rows == 3).all()


# widths of one element to many pieces, whole and odd
WIDTHS = [1, 8, 63, 64, 127, 128, 513, 1024, 2047, 4100]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T,picks,groups", [(1, 3, 4), (37, 2, 5), (700, 4, 33)])
@pytest.mark.parametrize("t", ["bfloat16", "float16", "float32"])
def test_sorted_rows(T, picks, groups, H, t):
    torch = torch_cuda()
    t = getattr(torch, t)
    e = experts_of(torch, T, picks, groups, H)
    x = normal(torch, (T, H), t, 1)
    for X in (x, padded(torch, x, 3, 1)):
        rows, order = lib.sgemm_grouped_sort(X, e, groups)
        offsets, _, source = check_order(torch, order, e, groups)
        kept = int(offsets[-1])
        assert torch.equal(rows[:kept], x[(source[:kept] // picks).cuda()])
        assert (rows[kept:] == 0).all() and rows.shape == (T * picks, H)


@pytest.mark.parametrize("T,picks,K", [(5, 3, 40), (300, 2, 1001), (2000, 4, 2047)])
def test_sorted_rows_in_8_bits(T, picks, K):
    torch = torch_cuda()
    e = experts_of(torch, T, picks, 6, K)
    x = lib.sgemm_i8_quantize(normal(torch, (T, K), torch.float32, 1))
    for X in (x, lib.I8Matrix(x.values.contiguous(), x.scales)):
        rows, order = lib.sgemm_grouped_sort(X, e, 6)
        offsets, _, source = check_order(torch, order, e, 6)
        kept = int(offsets[-1])
        at = (source[:kept] // picks).cuda()
        assert torch.equal(rows.values[:kept], x.values[at]) and torch.equal(rows.scales[:kept], x.scales[at])
        assert (rows.values[kept:] == 0).all() and (rows.scales[kept:] == 0).all()
        assert rows.values.stride(0) % 16 == 0


PAIRS = [("bfloat16", "bfloat16"), ("float16", "float16"), ("float32", "float32"), ("bfloat16", "float32"), ("float16", "float32"),
         ("float32", "bfloat16"), ("float32", "float16")]


def terms(torch, Y, position, weights):
    """weights * Y by (token, pick) in 64 bits, 0 for none."""
    live = position >= 0
    w = torch.ones(position.shape, dtype=torch.float64, device=Y.device) if weights is None else weights.double()
    return torch.where(live[..., None], Y.double()[position.clamp(min=0)] * torch.where(live, w, 0.0)[..., None], 0.0)


@pytest.mark.parametrize("H", [1, 40, 127, 128, 520, 2047, 4096])
@pytest.mark.parametrize("T,picks", [(1, 1), (3, 8), (130, 5), (2100, 3)])
@pytest.mark.parametrize("yt,ot", PAIRS)
def test_combine(T, picks, H, yt, ot):
    torch = torch_cuda()
    yt, ot = getattr(torch, yt), getattr(torch, ot)
    e = experts_of(torch, T, picks, 9, H)
    _, order = lib.sgemm_grouped_sort(None, e, 9)
    Y = normal(torch, (T * picks, H), yt, 1)
    Y[int(order.offsets[-1]):] = float("nan")           # rows of no group are not read
    position = order.position.long()
    for wt in (None, torch.float32, yt, torch.float16):
        w = None if wt is None else torch.rand(T, picks, generator=torch.Generator().manual_seed(2)).to(wt).cuda()
        if w is not None:
            w[position < 0] = float("inf")              # nor are their weights
        ref = terms(torch, Y, position, w)
        big = ref.abs().sum(1)
        tol = 2 * picks * 2 ** -24 * (1 + 2 ** -20) * big
        for V, W in ((Y, w), (padded(torch, Y, 5, 1), w if w is None else padded(torch, w, 2, 1))):
            got = lib.sgemm_grouped_combine(V, order, W, out_dtype=None if ot == yt else ot)
            assert got.dtype == ot and got.shape == (T, H)
            assert_within(torch, got, ref.sum(1), tol + u(ot, torch) * (ref.sum(1).abs() + tol) + torch.finfo(ot).tiny * torch.finfo(ot).eps)


@pytest.mark.parametrize("H", [1, 40, 127, 129, 520, 2047, 4096])
@pytest.mark.parametrize("T,picks", [(1, 1), (3, 9), (130, 5), (2100, 3)])
@pytest.mark.parametrize("yt,dt", PAIRS)
def test_combine_grad(T, picks, H, yt, dt):
    torch = torch_cuda()
    yt, dt = getattr(torch, yt), getattr(torch, dt)
    e = experts_of(torch, T, picks, 9, H)
    _, order = lib.sgemm_grouped_sort(None, e, 9)
    kept = int(order.offsets[-1])
    Y, D = normal(torch, (T * picks, H), yt, 1), normal(torch, (T, H), dt, 2)
    Y[kept:] = float("nan")
    position, source = order.position.long(), order.source.long()[:kept]
    live = position >= 0
    for wt in (None, torch.float32, yt):
        w = None if wt is None else torch.rand(T, picks, generator=torch.Generator().manual_seed(2)).to(wt).cuda()
        if w is not None:
            w[~live] = float("nan")
        for padding in (False, True):
            d, y = (padded(torch, D, 3, 1), padded(torch, Y, 5, 1)) if padding else (D, Y)
            dY, dw = lib.sgemm_grouped_combine_grad(d, y, order, w)
            assert dY.dtype == yt and dY.shape == Y.shape and (dY[kept:] == 0).all()
            rows = D.double()[source // picks]
            ref = rows if w is None else rows * w.double().reshape(-1)[source][:, None]
            assert_within(torch, dY[:kept], ref, (2 ** -24 + u(yt, torch)) * (1 + 2 ** -8) * ref.abs() + torch.finfo(yt).tiny * torch.finfo(yt).eps)
            if w is None:
                assert dw is None
                continue
            products = torch.where(live[..., None], Y.double()[position.clamp(min=0)], 0.0) * D.double()[:, None]
            ref, big = products.sum(2), products.abs().sum(2)
            assert dw.dtype == wt and dw.shape == (T, picks) and (dw[~live] == 0).all()
            tol = (H + 1) * 2 ** -24 * (1 + 2 ** -10) * big
            assert_within(torch, dw, ref, tol + u(wt, torch) * (ref.abs() + tol) + torch.finfo(wt).tiny)
    only = lib.sgemm_grouped_combine_grad(D, Y, order, w, need_dweights=False)
    assert only[1] is None and torch.equal(only[0], dY)
    only = lib.sgemm_grouped_combine_grad(D, Y, order, w, need_dy=False)
    assert only[0] is None and torch.equal(only[1], dw)


def test_gradients_against_differences():
    """The sum of G * combine(Y(X), w) with Y[r] = rows[r] * (1 + source): its
    directional derivatives along X and w by central differences."""
    torch = torch_cuda()
    T, picks, H, groups = 21, 3, 50, 5
    e = experts_of(torch, T, picks, groups, 1)
    X, w, G = (normal(torch, s, torch.float32, i) for i, s in enumerate([(T, H), (T, picks), (T, H)]))
    dX, dwts = normal(torch, (T, H), torch.float32, 7), normal(torch, (T, picks), torch.float32, 8)

    def value(X, w):
        rows, order = lib.sgemm_grouped_sort(X, e, groups)
        factor = (1 + order.source.clamp(min=0).float() / 7)[:, None]
        Y = rows * factor
        return (G.double() * lib.sgemm_grouped_combine(Y, order, w).double()).sum().item(), Y, order, factor

    base, Y, order, factor = value(X, w)
    dY, dw = lib.sgemm_grouped_combine_grad(G, Y, order, w)
    gX = lib.sgemm_grouped_combine(dY * factor, order)
    # the value is linear in X and in w, so a step of 1 has no error but the roundings of its terms: per term six to
    # FP32 (rows * factor, weights, sums of three) in each of two values and as many in the gradients, on terms that
    # the step makes up to 5 times as large (|X| + |dX| against |X|, in the sum): 18 * 5 < 128 roundings of `size`
    for along, a, b in (((gX.double() * dX).sum().item(), X + dX, X - dX), ((dw.double() * dwts).sum().item(), w + dwts, w - dwts)):
        hi, lo = (value(v, w)[0] if v.shape == X.shape else value(X, v)[0] for v in (a, b))
        size = (G.double().abs() * terms(torch, Y, order.position.long(), w).abs().sum(1)).sum().item()
        assert abs((hi - lo) / 2 - along) <= 128 * 2 ** -24 * size


def test_places_that_are_out_of_range():
    """Places outside the rows, in an order that did not come from the sort, are none."""
    torch = torch_cuda()
    T, picks, H = 40, 2, 33
    _, order = lib.sgemm_grouped_sort(None, experts_of(torch, T, picks, 3, 1, drop=0.0), 3)
    bad = order.position.clone()
    bad[3, 1], bad[4, 0], bad[5] = T * picks, -7, 2 ** 31 - 1
    Y, D, w = normal(torch, (T * picks, H), torch.float32, 1), normal(torch, (T, H), torch.float32, 2), torch.rand(T, picks, device="cuda")
    out = lib.sgemm_grouped_combine(Y, order._replace(position=bad), w)
    assert (out[5] == 0).all()
    ref = terms(torch, Y, torch.where((bad >= 0) & (bad < T * picks), bad, -1).long(), w)
    assert_within(torch, out, ref.sum(1), 8 * 2 ** -24 * ref.abs().sum(1))
    dY, dw = lib.sgemm_grouped_combine_grad(D, Y, order._replace(position=bad), w)
    assert (dw[5] == 0).all() and dw[4, 0] == 0 and dw[3, 1] == 0


@pytest.mark.parametrize("T,picks", [(16, 2), (1500, 4)])
def test_graph(T, picks):
    torch = torch_cuda()
    H, groups = 136, 10
    x = normal(torch, (T, H), torch.bfloat16, 1)
    e = experts_of(torch, T, picks, groups, 1)
    w = torch.rand(T, picks, device="cuda")

    def run():
        rows, order = lib.sgemm_grouped_sort(x, e, groups)
        out = lib.sgemm_grouped_combine(rows, order, w)
        dY, dw = lib.sgemm_grouped_combine_grad(out, rows, order, w)
        return [rows, *order, out, dY, dw]

    def refresh(i):
        x.copy_(normal(torch, (T, H), torch.bfloat16, 10 + i))
        e.copy_(experts_of(torch, T, picks, groups, 20 + i))
        w.copy_(torch.rand(T, picks, generator=torch.Generator().manual_seed(i)))

    def checked(outs, i):
        check_order(torch, lib.GroupOrder(*outs[1:4]), e, groups)
        for a, b in zip(outs, run()):
            assert torch.equal(a, b), i
    replays(torch, run, lambda o: o, refresh, checked)


def test_two_streams_and_a_given_one():
    torch = torch_cuda()
    x, e = normal(torch, (4000, 300), torch.float16, 1), experts_of(torch, 4000, 3, 20, 1)
    want, order = lib.sgemm_grouped_sort(x, e, 20)
    combined = lib.sgemm_grouped_combine(want, order)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(s, *lib.sgemm_grouped_sort(x, e, 20, stream=s)) for _ in range(4) for s in streams]
    back = [lib.sgemm_grouped_combine(rows, o, stream=s) for s, rows, o in got]
    torch.cuda.synchronize()
    assert all(torch.equal(rows, want) and torch.equal(b, combined) for (_, rows, _), b in zip(got, back))


def test_past_32_bits():
    """Rows of more than 2^32 bytes in all; the last lie behind."""
    torch = torch_cuda()
    T, picks, H, groups = 70000, 8, 4096, 16
    x = torch.randint(-8, 9, (T, H), device="cuda", dtype=torch.int8).bfloat16()
    e = torch.randint(0, groups, (T, picks), device="cuda")
    rows, order = lib.sgemm_grouped_sort(x, e, groups)
    assert torch.equal(rows[-1000:], x[order.source[-1000:].long() // picks])
    out = lib.sgemm_grouped_combine(rows, order)
    assert torch.equal(out[-1000:], x[-1000:] * picks) and torch.equal(out[:1000], x[:1000] * picks)
    del out
    w = torch.full((T, picks), 0.5, device="cuda")
    dY, dw = lib.sgemm_grouped_combine_grad(x, rows, order, w)
    assert torch.equal(dY[-1000:], rows[-1000:] * 0.5)
    assert torch.equal(dw[-1000:], (x[-1000:].double() ** 2).sum(1, keepdim=True).float().expand(-1, picks))


def test_refusals():
    torch = torch_cuda()
    X, e = torch.zeros(6, 8, device="cuda"), torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    for bad in (dict(X=X.double()), dict(X=X.char()), dict(experts=e.float()), dict(experts=e.short())):
        with pytest.raises(TypeError):
            lib.sgemm_grouped_sort(**{**dict(X=X, experts=e, groups=3), **bad})
    for bad in (dict(X=X[:5]), dict(X=X.cpu()), dict(experts=e.cpu()), dict(X=X.T.contiguous().T), dict(experts=e[None]), dict(groups=-1)):
        with pytest.raises(ValueError):
            lib.sgemm_grouped_sort(**{**dict(X=X, experts=e, groups=3), **bad})
    with pytest.raises(lib.SgemmError):
        lib.sgemm_grouped_sort(X, e, 4097)
    rows, order = lib.sgemm_grouped_sort(X, e, 3)
    w = torch.ones(6, 2, device="cuda")
    for bad in (dict(Y=rows[:11]), dict(Y=rows.cpu()), dict(weights=w.T), dict(weights=w.cpu()), dict(order=order._replace(position=order.position.cpu())),
                dict(order=order._replace(source=order.source[:4]))):
        with pytest.raises(ValueError):
            lib.sgemm_grouped_combine(**{**dict(Y=rows, order=order, weights=w), **bad})
        if "source" not in str(bad):
            with pytest.raises(ValueError):
                lib.sgemm_grouped_combine_grad(**{**dict(D=X, Y=rows, order=order, weights=w), **bad})
    for bad in (dict(Y=rows.half(), out_dtype=torch.bfloat16), dict(Y=rows.double()), dict(weights=w.double()), dict(order=order._replace(offsets=order.offsets.long()))):
        with pytest.raises(TypeError):
            lib.sgemm_grouped_combine(**{**dict(Y=rows, order=order, weights=w), **bad})


@pytest.mark.parametrize("T", [5, 3000])
def test_scales_of_rows_without_columns(T):
    """8-bit rows of no columns have scales, which are brought to their places too."""
    torch = torch_cuda()
    picks, groups = 2, 3
    e = experts_of(torch, T, picks, groups, 1)
    x = lib.I8Matrix(torch.zeros(T, 0, dtype=torch.int8, device="cuda"), torch.arange(1.0, T + 1, device="cuda"))
    rows, order = lib.sgemm_grouped_sort(x, e, groups)
    offsets, _, source = check_order(torch, order, e, groups)
    kept = int(offsets[-1])
    want = torch.zeros(T * picks, device="cuda")
    want[:kept] = x.scales[(source[:kept] // picks).cuda()]
    assert rows.values.shape == (T * picks, 0) and torch.equal(rows.scales, want)
    held = torch.full((T * picks,), float("nan"), device="cuda")
    offsets, position, source = (torch.zeros_like(o) for o in order)
    ws = torch.empty(max(lib.capi.sgemm_grouped_sort_workspace(T, picks, groups), 16), dtype=torch.uint8, device="cuda")
    st = lib.capi.sgemm_grouped_sort(lib.capi.SGEMM_DTYPE_I8, T, picks, groups, 0, None, 1, x.scales.data_ptr(), e.data_ptr(), picks,
                                     e.element_size(), offsets.data_ptr(), position.data_ptr(), source.data_ptr(), None, 1, held.data_ptr(),
                                     ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == lib.capi.SGEMM_STATUS_OK and torch.equal(held, want)

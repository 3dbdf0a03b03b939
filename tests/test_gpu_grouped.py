"""sgemm_grouped and sgemm_grouped_wgrad against 64-bit products."""
import pytest

import fp32_sgemm_tuning_amd as lib
from fp32_sgemm_tuning_amd import capi
from gpu_util import torch_cuda
from products_util import (assert_equal, assert_within, grouped_ref, ints, normal, padded, replays, u, wgrad_ref)

pytestmark = pytest.mark.gpu

# (rows, offsets): empty groups first, last and between, single rows, rows of
# no group before, behind; more groups than a wave has lanes
SPLITS = {
    "one row": (1, [0, 1]),
    "one group": (129, [0, 129]),
    "single rows": (5, [0, 1, 2, 3, 4, 5]),
    "empty ends": (300, [0, 0, 140, 140, 141, 300, 300]),
    "rows of no group": (200, [7, 20, 20, 150]),
    "no rows": (40, [13, 13, 13]),
    "even": (512, [0, 128, 256, 384, 512]),
    "one large": (700, [0, 3, 690, 691, 700]),
    "many groups": (333, [min(333, i * 333 // 150 + (i % 3)) for i in range(150)] + [333]),
    "more groups than rows": (3, [0, 0, 1, 1, 1, 2, 2, 3, 3, 3]),
}
SIZES = [(64, 128), (8, 8), (200, 264), (1, 1), (37, 131), (72, 5), (1000, 130)]
KINDS = [("bfloat16", "float32", False), ("bfloat16", "bfloat16", True), ("float16", "float16", False),
         ("float16", "float32", True)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("K,N", SIZES)
def test_rows_exact(split, K, N, kind):
    torch = torch_cuda()
    T, off = SPLITS[split]
    dtype, out, tb = getattr(torch, kind[0]), getattr(torch, kind[1]), kind[2]
    G = len(off) - 1
    A = ints(torch, (T, K), -3, 3, dtype, 1)
    B = ints(torch, (G, N, K) if tb else (G, K, N), -3, 3, dtype, 2)
    ref, live = grouped_ref(torch, A, B, off, tb)
    A[~live] = float("nan")                       # rows of no group are not read into any result
    C = torch.full((T, N), 7.0, dtype=out, device="cuda")
    got = lib.sgemm_grouped(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), C=C, trans_b=tb)
    torch.cuda.synchronize()
    assert got is C
    ref[~live] = 7.0
    assert_equal(torch, C, ref, split)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("K,N", SIZES)
def test_wgrad_exact(split, K, N, kind):
    torch = torch_cuda()
    T, off = SPLITS[split]
    dtype, out = getattr(torch, kind[0]), getattr(torch, kind[1])
    A, D = ints(torch, (T, K), -3, 3, dtype, 3), ints(torch, (T, N), -3, 3, dtype, 4)
    ref = wgrad_ref(torch, A, D, off)
    for x in (A, D):
        x[:off[0]] = float("nan")
        x[off[-1]:] = float("nan")
    got = lib.sgemm_grouped_wgrad(A, D, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out)
    torch.cuda.synchronize()
    assert_equal(torch, got, ref, split)


@pytest.mark.parametrize("T,G,K,N", [(4000, 4, 264, 520), (4097, 7, 512, 1000), (2600, 3, 1032, 4104), (640, 16, 264, 1000)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_larger(T, G, K, N, dtype):
    """The larger tiles, and sums of normal values against the bound."""
    torch = torch_cuda()
    dtype = getattr(torch, dtype)
    off = sorted((torch.randint(0, T + 1, (G - 1,), generator=torch.Generator().manual_seed(T))).tolist())
    off = [0] + off + [T]
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    A, D = normal(torch, (T, K), dtype, 5), normal(torch, (T, N), dtype, 6)
    B = normal(torch, (G, K, N), dtype, 7)
    ref, _ = grouped_ref(torch, A, B, off, False)
    big, _ = grouped_ref(torch, A.abs(), B.abs(), off, False)
    assert_within(torch, lib.sgemm_grouped(A, B, dev), ref, (K + 1) * 2 ** -23 * big, "rows")
    ref, _ = grouped_ref(torch, D, B, off, True)
    big, _ = grouped_ref(torch, D.abs(), B.abs(), off, True)
    assert_within(torch, lib.sgemm_grouped(D, B, dev, trans_b=True, out_dtype=dtype), ref,
                  (N + 1) * 2 ** -23 * big + 1.01 * u(dtype, torch) * ref.abs() + 2 ** -25, "rows, 16 bits")
    ref, big = wgrad_ref(torch, A, D, off), wgrad_ref(torch, A.abs(), D.abs(), off)
    assert_within(torch, lib.sgemm_grouped_wgrad(A, D, dev), ref, (T + 1) * 2 ** -23 * big, "wgrad")


@pytest.mark.parametrize("off", [[0, 3000, 6000], [0, 5999, 6000], [100, 100, 5000], [0, 6000]], ids=str)
@pytest.mark.parametrize("K,N", [(72, 40), (5, 131), (264, 200)])
@pytest.mark.parametrize("out", ["float32", "bfloat16"])
def test_small_matrices_over_many_rows(K, N, off, out):
    """The weight gradient summed in shares of the rows; beta joins in once."""
    torch = torch_cuda()
    A, D = ints(torch, (6000, K), -2, 2, torch.bfloat16, 3), ints(torch, (6000, N), -2, 2, torch.bfloat16, 4)
    C = ints(torch, (len(off) - 1, K, N), -8, 8, getattr(torch, out), 5)
    want = 0.5 * wgrad_ref(torch, A, D, off) + 2 * C.double()
    A[:off[0]], A[off[-1]:] = float("nan"), float("nan")
    lib.sgemm_grouped_wgrad(A, D, torch.tensor(off, dtype=torch.int32, device="cuda"), C=C, alpha=0.5, beta=2.0)
    assert_equal(torch, C, want)


@pytest.mark.parametrize("out", ["float32", "float16"])
@pytest.mark.parametrize("pads", [(8, 16, 4, 0), (3, 1, 1, 0), (8, 8, 2, 1), (0, 0, 3, 8)])
def test_strides_alpha_beta(pads, out):
    """Padded rows, unaligned bases, a strided C; alpha and beta; nothing
    outside the views is read into a result or written."""
    torch = torch_cuda()
    pa, pb, pc, base = pads
    T, G, K, N = 150, 3, 72, 136
    off = [0, 60, 61, 140]
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    A, B = ints(torch, (T, K), -2, 2, torch.float16, 1), ints(torch, (G, K, N), -2, 2, torch.float16, 2)
    D = ints(torch, (T, N), -2, 2, torch.float16, 3)
    C0 = ints(torch, (T, N), -8, 8, getattr(torch, out), 4)
    E0 = ints(torch, (G, K, N), -8, 8, getattr(torch, out), 5)
    Av, Bv, Dv = padded(torch, A, pa, base), padded(torch, B, pb, base), padded(torch, D, pb, base)
    Cv, Ev = padded(torch, C0, pc, base, fill=99.0), padded(torch, E0, pc, base, fill=99.0)
    lib.sgemm_grouped(Av, Bv, dev, C=Cv, alpha=0.5, beta=-2.0)
    lib.sgemm_grouped_wgrad(Av, Dv, dev, C=Ev, alpha=2.0, beta=0.5)
    torch.cuda.synchronize()
    ref, live = grouped_ref(torch, A, B, off, False)
    want = torch.where(live[:, None], 0.5 * ref - 2 * C0.double(), C0.double())
    assert_equal(torch, Cv, want)
    assert_equal(torch, Ev, 2 * wgrad_ref(torch, A, D, off) + 0.5 * E0.double())
    for v, rows in ((Cv, T), (Ev, G * K)):
        whole = torch.as_strided(v, (rows, N + pc), (N + pc, 1))
        assert (whole[:, N:] == 99.0).all()


def test_beta_zero_reads_nothing():
    torch = torch_cuda()
    A, B = ints(torch, (40, 64), -2, 2, torch.bfloat16, 1), ints(torch, (2, 64, 64), -2, 2, torch.bfloat16, 2)
    dev = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    C = torch.full((40, 64), float("nan"), device="cuda")
    E = torch.full((2, 64, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.sgemm_grouped(A, B, dev, C=C)
    lib.sgemm_grouped_wgrad(A, A, dev, C=E)
    assert not C.isnan().any() and not E.isnan().any()


def test_shared_and_transposed_weights():
    """One matrix for all groups (batch stride 0)."""
    torch = torch_cuda()
    A, W = ints(torch, (100, 48), -2, 2, torch.bfloat16, 1), ints(torch, (40, 48), -2, 2, torch.bfloat16, 2)
    off = [0, 30, 100]
    got = lib.sgemm_grouped(A, W.expand(2, 40, 48), torch.tensor(off, dtype=torch.int32, device="cuda"), trans_b=True)
    assert_equal(torch, got, A.double() @ W.double().T.contiguous())


def test_nan_stays_in_its_row_and_group():
    torch = torch_cuda()
    off = [0, 50, 90, 200]
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    A, B = ints(torch, (200, 64), -2, 2, torch.bfloat16, 1), ints(torch, (3, 64, 72), -2, 2, torch.bfloat16, 2)
    ref, _ = grouped_ref(torch, A, B, off, False)
    dref = wgrad_ref(torch, A, A, off)
    A[60] = float("nan")
    got = lib.sgemm_grouped(A, B, dev)
    assert got[60].isnan().all()
    keep = torch.arange(200, device="cuda") != 60
    assert_equal(torch, got[keep], ref[keep])
    dgot = lib.sgemm_grouped_wgrad(A, A, dev)
    assert dgot[1].isnan().all()
    assert_equal(torch, dgot[0], dref[0])
    assert_equal(torch, dgot[2], dref[2])


def test_no_inner_extent_and_no_groups():
    torch = torch_cuda()
    dev = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    e = torch.bfloat16
    C = torch.full((6, 16), 3.0, device="cuda")
    lib.sgemm_grouped(torch.empty(6, 0, dtype=e, device="cuda"), torch.empty(2, 0, 16, dtype=e, device="cuda"), dev, C=C,
                      beta=2.0)
    assert (C[:5] == 6).all() and (C[5] == 3).all()
    got = lib.sgemm_grouped_wgrad(torch.empty(0, 8, dtype=e, device="cuda"), torch.empty(0, 16, dtype=e, device="cuda"),
                                  torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert got.shape == (2, 8, 16) and (got == 0).all()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    C = torch.full((6, 16), 3.0, device="cuda")
    lib.sgemm_grouped(torch.ones(6, 8, dtype=e, device="cuda"), torch.empty(0, 8, 16, dtype=e, device="cuda"), none, C=C)
    assert (C == 3).all()
    assert lib.sgemm_grouped_wgrad(torch.ones(6, 8, dtype=e, device="cuda"), torch.ones(6, 8, dtype=e, device="cuda"),
                                   none).shape == (0, 8, 8)


def test_offsets_outside_are_clamped():
    torch = torch_cuda()
    A, B = ints(torch, (70, 64), -2, 2, torch.bfloat16, 1), ints(torch, (3, 64, 64), -2, 2, torch.bfloat16, 2)
    dev = torch.tensor([-5, 30, 90, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    ref, _ = grouped_ref(torch, A, B, [0, 30, 70, 70], False)
    assert_equal(torch, lib.sgemm_grouped(A, B, dev), ref)
    assert_equal(torch, lib.sgemm_grouped_wgrad(A, A, dev), wgrad_ref(torch, A, A, [0, 30, 70, 70]))


def test_gradients_against_differences():
    """sum(R * C) is linear in A and in B, so its central differences along a
    direction are the gradients' products with it, exactly but for rounding:
    integer inputs make both sides exact."""
    torch = torch_cuda()
    e, off = torch.bfloat16, [0, 9, 9, 40, 77]
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    A, B, R = ints(torch, (77, 24), -2, 2, e, 1), ints(torch, (4, 24, 40), -2, 2, e, 2), ints(torch, (77, 40), -2, 2, e, 3)
    dA = lib.sgemm_grouped(R, B, dev, trans_b=True).double()
    dB = lib.sgemm_grouped_wgrad(A, R, dev).double()

    def value(a, b):
        return (grouped_ref(torch, a, b, off, False)[0] * R.double()).sum()
    vA, vB = ints(torch, A.shape, -1, 1, e, 4), ints(torch, B.shape, -1, 1, e, 5)
    assert (dA * vA.double()).sum() == (value(A + vA, B) - value(A - vA, B)) / 2
    assert (dB * vB.double()).sum() == (value(A, B + vB) - value(A, B - vB)) / 2


def test_captured_with_new_offsets():
    torch = torch_cuda()
    A, B = ints(torch, (260, 72), -2, 2, torch.float16, 1), ints(torch, (3, 72, 100), -2, 2, torch.float16, 2)
    dev = torch.tensor([0, 50, 60, 260], dtype=torch.int32, device="cuda")
    offs = [[0, 0, 130, 260], [10, 200, 200, 250], [0, 1, 2, 3]]

    def run():
        return lib.sgemm_grouped(A, B, dev), lib.sgemm_grouped_wgrad(A, A, dev)

    def check(outs, i):
        ref, live = grouped_ref(torch, A, B, offs[i], False)
        assert_equal(torch, outs[0][live], ref[live], f"replay {i}")
        assert (outs[0][~live] == 0).all()
        assert_equal(torch, outs[1], wgrad_ref(torch, A, A, offs[i]), f"replay {i}")
        assert_equal(torch, lib.sgemm_grouped(A, B, dev)[live], ref[live], "eager beside it")
    replays(torch, run, lambda o: o, lambda i: dev.copy_(torch.tensor(offs[i], dtype=torch.int32)), check)


def test_two_streams_at_once():
    torch = torch_cuda()
    cases = []
    for i in range(2):
        A, B = ints(torch, (900, 131), -2, 2, torch.bfloat16, i), ints(torch, (4, 131, 257), -2, 2, torch.bfloat16, 9 + i)
        off = [0, 100 + i, 400, 401, 900]
        cases.append((A, B, off, torch.tensor(off, dtype=torch.int32, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[lib.sgemm_grouped(A, B, dev, stream=s) for A, B, _, dev, s in cases] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in outs:
        for got, (A, B, off, _, _) in zip(pair, cases):
            assert_equal(torch, got, grouped_ref(torch, A, B, off, False)[0])


def test_race_check_build(monkeypatch):
    """The same products with LDS stages poisoned between their last read and
    their refill."""
    torch = torch_cuda()
    monkeypatch.setattr(capi, "_lib", capi.open_library(capi.POISON_LIB_PATH))
    for T, K, N in ((60, 200, 264), (900, 264, 392), (3000, 520, 520), (5000, 72, 136)):
        off = [0, T // 3, T // 2, T]
        dev = torch.tensor(off, dtype=torch.int32, device="cuda")
        A, B = ints(torch, (T, K), -3, 3, torch.bfloat16, 1), ints(torch, (3, K, N), -3, 3, torch.bfloat16, 2)
        D = ints(torch, (T, N), -3, 3, torch.bfloat16, 3)
        for got, ref in ((lib.sgemm_grouped(A, B, dev), grouped_ref(torch, A, B, off, False)[0]),
                         (lib.sgemm_grouped(D, B, dev, trans_b=True), grouped_ref(torch, D, B, off, True)[0]),
                         (lib.sgemm_grouped_wgrad(A, D, dev), wgrad_ref(torch, A, D, off))):
            assert_equal(torch, got, ref, f"{T} rows")


def test_refusals():
    torch = torch_cuda()
    e = torch.bfloat16
    A, B = torch.ones(6, 8, dtype=e, device="cuda"), torch.ones(2, 8, 16, dtype=e, device="cuda")
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    D = torch.ones(6, 16, dtype=e, device="cuda")
    for bad in (dict(A=A.float()), dict(A=A.half()), dict(offsets=off.long()), dict(out_dtype=torch.float16),
                dict(C=torch.ones(6, 16, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            lib.sgemm_grouped(**{**dict(A=A, B=B, offsets=off), **bad})
    for bad in (dict(B=B[:1]), dict(trans_b=True), dict(offsets=off[:2]), dict(offsets=off[None]), dict(A=A[0]),
                dict(A=A.T), dict(C=torch.ones(5, 16, device="cuda")), dict(beta=1.0), dict(A=A.cpu()),
                dict(offsets=off.cpu()), dict(offsets=off[::2])):
        with pytest.raises(ValueError):
            lib.sgemm_grouped(**{**dict(A=A, B=B, offsets=off), **bad})
    with pytest.raises(ValueError):
        lib.sgemm_grouped_wgrad(A, D[:5], off)
    with pytest.raises(TypeError):
        lib.sgemm_grouped_wgrad(A, D.half(), off)
    with pytest.raises(ValueError):
        lib.sgemm_grouped_wgrad(A, D, off, C=torch.ones(2, 16, 8, device="cuda"))
    with pytest.raises(lib.SgemmError) as err:      # groups that overlap in C
        lib.sgemm_grouped_wgrad(A, D, off, C=torch.ones(1, 8, 16, device="cuda").expand(2, 8, 16))
    assert err.value.status == capi.SGEMM_STATUS_INVALID_DIM

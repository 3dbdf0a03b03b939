"""Limits of the grouped products, the output layer with its loss and the
4-bit weights that show without a device: every call below returns before any
HIP call."""
import pytest

from fp32_sgemm_tuning_amd import capi
from test_products_cpu import DIM, GROUPED, NULL, W4, WGRAD, XENT
from w4_forms import FORMS, SHAPES

AL = 0x10000                        # a fake device address, aligned; never dereferenced


@pytest.mark.parametrize("M", range(1, 9))
@pytest.mark.parametrize("N", [17_180_000, 1 << 25, 1 << 26, 1 << 28, 1 << 30])
def test_pieces_of_a_large_vocabulary_fit_a_descriptor(M, N):
    """P [M, piece] is the transposed operand of dW: its descriptor spans up to
    63 rows of it and 256 columns, which must end below the 2^31 that stands
    for "out of range".  (The workspace bounds the piece's columns from above.)"""
    columns = capi.sgemm_lowp_xent_workspace(M, N, 8, AL, 8, AL, 8, 1) // (2 * M)
    assert 2 * (63 * columns + 256) <= 1 << 31


@pytest.mark.parametrize("form,M,N", SHAPES)
def test_form_of_a_4bit_product(form, M, N):
    """The shapes the 4-bit products are tested on take every launch form."""
    assert capi.sgemm_w4_select_form(M, N) == form


def test_forms_of_4bit_products():
    assert {f for f, _, _ in SHAPES} == set(FORMS)
    seen = {capi.sgemm_w4_select_form(M, N) for M in (1, 16, 17, 64, 65, 100, 128, 256, 1000, 4096)
            for N in (1, 100, 3200, 4096, 6400, 8192, 12800, 14336, 50000)}
    assert seen == set(FORMS)
    for bad in ((-1, 5), (5, -1)):
        assert capi.sgemm_w4_select_form(*bad) == capi.SGEMM_STATUS_INVALID_DIM


@pytest.mark.parametrize("call,good,fits,over", [
    # tiles of 256 x 256, and 256 workgroups for the last round: 2^23 of 512 threads are one too many
    (capi.sgemm_lowp_grouped, {**GROUPED, "C": None}, dict(M=2 ** 31 - 1 - (1 << 18)), dict(M=2 ** 31 - 1)),
    (capi.sgemm_lowp_grouped, {**GROUPED, "C": None}, dict(M=1 << 24, N=30000, ldb=30000, ldc=30000),
     dict(M=1 << 24, N=40000, ldb=40000, ldc=40000)),
    # small groups, tiles of 32 x 128
    (capi.sgemm_lowp_grouped, {**GROUPED, "C": None}, dict(M=60000, groups=60000, N=30000, ldb=30000, ldc=30000),
     dict(M=60000, groups=60000, N=40000, ldb=40000, ldc=40000)),
    (capi.sgemm_lowp_grouped_wgrad, {**WGRAD, "C": None}, dict(groups=1000, K=1, N=1 << 20, ldd=1 << 20, ldc=1 << 20, stride_c=1 << 20),
     dict(groups=1100, K=1, N=1 << 20, ldd=1 << 20, ldc=1 << 20, stride_c=1 << 20)),
    (capi.sgemm_lowp_xent, {**XENT, "loss": None}, dict(M=1 << 24, N=32512), dict(M=1 << 24, N=32768)),
    (capi.sgemm_lowp_xent, {**XENT, "loss": None}, dict(M=32, N=1 << 30), dict(M=1024, N=1 << 30)),
    (capi.sgemm_w4, {**W4, "C": None}, dict(M=1, N=2 ** 29 - 64, ldc=1 << 30), dict(M=1, N=1 << 29, ldc=1 << 30)),
    (capi.sgemm_w4, {**W4, "C": None}, dict(M=1 << 24, N=4096, ldc=1 << 30), dict(M=1 << 24, N=1 << 16, ldc=1 << 30)),
], ids=lambda v: getattr(v, "__name__", ""))
def test_results_of_more_tiles_than_a_launch_covers(call, good, fits, over):
    """Refused before anything is enqueued; what fits goes on to the next
    check (a missing result)."""
    assert call(**{**good, **fits}) == NULL
    assert call(**{**good, **over}) == DIM


@pytest.mark.parametrize("status,names", [
    (capi.SGEMM_STATUS_UNSUPPORTED, ["variant", "16-byte aligned pointers and leading dimensions", "packed 16-byte", "scales 8-byte", "zeros 4-byte"]),
    (capi.SGEMM_STATUS_INVALID_DTYPE, ["SGEMM_DTYPE_BF16", "SGEMM_DTYPE_F16", "SGEMM_DTYPE_F32"]),
    (capi.SGEMM_STATUS_SCRATCH_TOO_SMALL, ["sgemm_noalloc", "SGEMM_NOALLOC_SCRATCH_BYTES", "workspace", "16-byte aligned"])])
def test_error_texts_name_what_is_wrong(status, names):
    """A status that several calls share says for each what it stands for."""
    text = capi.sgemm_strerror(status)
    assert all(n in text for n in names), text


def test_sizes_past_an_int_are_refused():
    """ctypes keeps the low 32 bits of an int argument: a row stride of 2^32 + 64
    would be read as 64."""
    import torch

    import fp32_sgemm_tuning_amd as lib
    e = torch.bfloat16

    def far(rows, cols, step, dtype=e):                 # (no memory behind it)
        return torch.empty(0, dtype=dtype, device="meta").as_strided((rows, cols), (step, 1))

    x, off = far(4, 64, 64), torch.empty(3, dtype=torch.int32, device="meta")
    t, v = torch.empty(4, dtype=torch.int64, device="meta"), torch.empty(4, device="meta")
    bad, tall = far(4, 64, 2 ** 32 + 64), far(2 ** 32 + 4, 64, 64)
    big = torch.empty(0, dtype=e, device="meta").as_strided((2, 64, 8), (0, 2 ** 32 + 8, 1))
    w4 = lib.W4Weight(torch.empty(2 ** 32 + 8, 64, dtype=torch.uint8, device="meta"),
                      torch.empty(2 ** 32 + 8, 1, dtype=e, device="meta"), None, 64, 128)
    calls = [lambda: lib.sgemm_grouped(bad, torch.empty(2, 64, 8, dtype=e, device="meta"), off),
             lambda: lib.sgemm_grouped(tall, torch.empty(2, 64, 8, dtype=e, device="meta"), off),
             lambda: lib.sgemm_grouped(x, big, off),
             lambda: lib.sgemm_grouped_wgrad(x, bad, off), lambda: lib.sgemm_xent(x, bad, t),
             lambda: lib.sgemm_xent(x, tall, t),
             lambda: lib.sgemm_xent_grad(x, x, t, v, torch.empty(0, device="meta").as_strided((4,), (2 ** 32 + 1,))),
             lambda: lib.sgemm_w4(x, w4), lambda: lib.sgemm_w4_dequantize(w4), lambda: lib.sgemm_w4_quantize(bad),
             lambda: lib._result(far(4, 8, 2 ** 32 + 8, torch.float32), (4, 8), None, x)]
    lib._codes()
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()

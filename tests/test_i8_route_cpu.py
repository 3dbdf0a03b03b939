"""Argument checks of the 8-bit products and of the sorting and combining of
rows: every call below returns before any HIP call."""
import pytest

from fp32_sgemm_tuning_amd import capi

AL, MIS = 0x10000, 0x10002          # fake device addresses, aligned and not; never dereferenced

I8 = dict(M=17, N=32, K=64, alpha=1.0, X=AL, ldx=64, x_scales=AL, W=AL, ldw=64, w_scales=AL, beta=0.0, C=AL, ldc=32, dtype_c=1,
          workspace=None, workspace_bytes=0, stream=None)
GROUPED = dict(groups=2, M=64, N=32, K=64, alpha=1.0, X=AL, ldx=64, x_scales=AL, W=AL, ldw=64, stride_w=2048, w_scales=AL, stride_s=32,
               offsets=AL, beta=0.0, C=AL, ldc=32, dtype_c=3, workspace=None, workspace_bytes=0, stream=None)
QUANT = dict(dtype=1, M=3, K=40, X=AL, ldx=40, values=AL, ldv=48, scales=AL, stream=None)
DEQUANT = dict(dtype=3, M=3, K=40, values=AL, ldv=48, scales=AL, X=AL, ldx=40, stream=None)
SORT = dict(dtype=1, T=10, picks=2, groups=4, H=16, X=AL, ldx=16, x_scales=None, experts=AL, lde=2, expert_bytes=8, offsets=AL, position=AL,
            source=AL, rows=AL, ldr=16, row_scales=None, workspace=None, workspace_bytes=0, stream=None)
COMBINE = dict(dtype=1, dtype_out=3, T=10, picks=2, H=16, Y=AL, ldy=16, position=AL, weights=AL, ldw=2, dtype_w=3, out=AL, ldo=16, stream=None)
GRAD = dict(dtype=1, dtype_d=1, T=10, picks=2, groups=4, H=16, D=AL, ldd=16, Y=AL, ldy=16, offsets=AL, position=AL, weights=AL, ldw=2, dtype_w=2,
            dY=AL, lddy=16, dweights=AL, stream=None)

DIM, NULL, TYPE, SMALL, OK = (capi.SGEMM_STATUS_INVALID_DIM, capi.SGEMM_STATUS_NULL_POINTER, capi.SGEMM_STATUS_INVALID_DTYPE,
                              capi.SGEMM_STATUS_SCRATCH_TOO_SMALL, capi.SGEMM_STATUS_OK)

REFUSED = [
    (capi.sgemm_i8, I8, [
        (TYPE, dict(dtype_c=0)), (TYPE, dict(dtype_c=4)), (DIM, dict(M=-1)), (DIM, dict(N=-1)), (DIM, dict(K=-1)), (DIM, dict(ldx=63)),
        (DIM, dict(ldw=63)), (DIM, dict(ldc=31)), (DIM, dict(K=1 << 17, ldx=1 << 17, ldw=1 << 17)), (DIM, dict(M=(1 << 24) + 1)),
        (DIM, dict(N=(1 << 30) + 1, ldc=2 ** 31 - 1)), (DIM, dict(M=1 << 24, N=1 << 16, ldc=1 << 16)),
        (NULL, dict(X=None)), (NULL, dict(W=None)), (NULL, dict(C=None)), (NULL, dict(x_scales=None)), (NULL, dict(w_scales=None)),
        (SMALL, dict(X=MIS)), (SMALL, dict(W=AL + 8)), (SMALL, dict(ldx=65)), (SMALL, dict(ldw=72)),
        (SMALL, dict(ldx=65, workspace=AL, workspace_bytes=17 * 64 - 1)), (SMALL, dict(X=MIS, workspace=MIS, workspace_bytes=1 << 30))]),
    (capi.sgemm_i8_grouped, GROUPED, [
        (TYPE, dict(dtype_c=4)), (DIM, dict(groups=-1)), (DIM, dict(groups=65535)), (DIM, dict(M=-1)), (DIM, dict(N=-1)), (DIM, dict(K=-1)),
        (DIM, dict(ldx=63)), (DIM, dict(ldw=63)), (DIM, dict(ldc=31)), (DIM, dict(stride_w=-1)), (DIM, dict(stride_s=-1)),
        (DIM, dict(K=1 << 17, ldx=1 << 17, ldw=1 << 17)), (DIM, dict(M=2 ** 31 - 1, N=1 << 21, ldc=1 << 21)),
        (DIM, dict(M=60000, groups=60000, N=40000, ldc=40000)),
        (NULL, dict(X=None)), (NULL, dict(W=None)), (NULL, dict(C=None)), (NULL, dict(x_scales=None)), (NULL, dict(w_scales=None)),
        (NULL, dict(offsets=None)), (SMALL, dict(X=MIS)), (SMALL, dict(stride_w=2049)), (SMALL, dict(ldw=65, stride_w=2080)),
        (SMALL, dict(ldw=65, stride_w=2080, workspace=AL, workspace_bytes=2 * 32 * 64 - 1))]),
    (capi.sgemm_i8_quantize, QUANT, [
        (TYPE, dict(dtype=0)), (TYPE, dict(dtype=4)), (DIM, dict(M=-1)), (DIM, dict(K=-1)), (DIM, dict(ldx=39)), (DIM, dict(ldv=39)),
        (DIM, dict(M=1 << 24, K=2000, ldx=2000, ldv=2000)), (DIM, dict(M=1 << 28)),
        (DIM, dict(K=(1 << 30) + 1, ldx=2 ** 31 - 1, ldv=2 ** 31 - 1)), (NULL, dict(X=None)), (NULL, dict(values=None)), (NULL, dict(scales=None))]),
    (capi.sgemm_i8_dequantize, DEQUANT, [
        (TYPE, dict(dtype=4)), (DIM, dict(M=-1)), (DIM, dict(K=-1)), (DIM, dict(ldx=39)), (DIM, dict(ldv=39)),
        (DIM, dict(K=(1 << 30) + 1, ldx=2 ** 31 - 1, ldv=2 ** 31 - 1)), (NULL, dict(X=None)), (NULL, dict(values=None)), (NULL, dict(scales=None))]),
    (capi.sgemm_grouped_sort, SORT, [
        (TYPE, dict(dtype=0)), (TYPE, dict(dtype=5)), (TYPE, dict(expert_bytes=2)), (DIM, dict(T=-1)), (DIM, dict(picks=-1, lde=2)), (DIM, dict(groups=-1)),
        (DIM, dict(groups=4097)), (DIM, dict(H=-1)), (DIM, dict(ldx=15)), (DIM, dict(ldr=15)), (DIM, dict(lde=1)), (DIM, dict(T=1 << 30)),
        (DIM, dict(H=(1 << 28) + 1, ldx=1 << 29, ldr=1 << 29)),
        (NULL, dict(X=None)), (NULL, dict(experts=None)), (NULL, dict(offsets=None)), (NULL, dict(position=None)), (NULL, dict(source=None)),
        (NULL, dict(dtype=4)), (NULL, dict(dtype=4, x_scales=AL)), (NULL, dict(T=0, offsets=None)),
        (SMALL, dict(T=3000)), (SMALL, dict(T=3000, workspace=AL, workspace_bytes=12 * 5 * 4 - 1)), (SMALL, dict(T=3000, workspace=MIS, workspace_bytes=1 << 30))]),
    (capi.sgemm_grouped_combine, COMBINE, [
        (TYPE, dict(dtype=4)), (TYPE, dict(dtype_out=2)), (TYPE, dict(dtype_w=4)), (DIM, dict(T=-1)), (DIM, dict(picks=-1)), (DIM, dict(H=-1)),
        (DIM, dict(ldy=15)), (DIM, dict(ldo=15)), (DIM, dict(ldw=1)), (DIM, dict(T=1 << 30)), (NULL, dict(Y=None)), (NULL, dict(position=None)),
        (NULL, dict(out=None))]),
    (capi.sgemm_grouped_combine_grad, GRAD, [
        (TYPE, dict(dtype=4)), (TYPE, dict(dtype_d=2)), (TYPE, dict(dtype_w=0)), (TYPE, dict(weights=None, dtype_w=0)), (DIM, dict(T=-1)), (DIM, dict(groups=-1)),
        (DIM, dict(ldd=15)), (DIM, dict(ldy=15)), (DIM, dict(lddy=15)), (DIM, dict(ldw=1)), (NULL, dict(D=None)), (NULL, dict(Y=None)),
        (NULL, dict(offsets=None)), (NULL, dict(position=None))]),
]


@pytest.mark.parametrize("call,good,want,bad", [(c, g, w, b) for c, g, cases in REFUSED for w, b in cases],
                         ids=lambda v: getattr(v, "__name__", None) or (str(v)[:40] if isinstance(v, dict) and len(v) < 8 else ""))
def test_refused(call, good, want, bad):
    assert call(**{**good, **bad}) == want


@pytest.mark.parametrize("call,good,empty", [
    (capi.sgemm_i8, I8, dict(M=0)), (capi.sgemm_i8, I8, dict(N=0)), (capi.sgemm_i8_grouped, GROUPED, dict(M=0)),
    (capi.sgemm_i8_grouped, GROUPED, dict(N=0)), (capi.sgemm_i8_grouped, GROUPED, dict(groups=0)), (capi.sgemm_i8_quantize, QUANT, dict(M=0)),
    (capi.sgemm_i8_dequantize, DEQUANT, dict(M=0)), (capi.sgemm_i8_dequantize, DEQUANT, dict(K=0)), (capi.sgemm_grouped_combine, COMBINE, dict(T=0)),
    (capi.sgemm_grouped_combine, COMBINE, dict(H=0)), (capi.sgemm_grouped_combine_grad, GRAD, dict(T=0)),
    (capi.sgemm_grouped_combine_grad, GRAD, dict(picks=0)), (capi.sgemm_grouped_combine_grad, GRAD, dict(dY=None, dweights=None))])
def test_empty_calls_launch_nothing(call, good, empty):
    assert call(**{**good, **empty}) == OK


def test_workspaces():
    ws = capi.sgemm_i8_workspace
    assert ws(3, 32, 64, AL, 64, AL, 64) == 0
    assert ws(3, 32, 61, AL, 64, AL, 64) == 0                   # what lies behind K is not used
    assert ws(20, 32, 61, AL, 61, AL, 64) == 1280               # 20 rows of 64 bytes, whole 256s
    assert ws(20, 32, 61, AL, 61, AL + 1, 64) == 1280 + 2048
    assert ws(16, 50000, 61, AL, 61, AL + 1, 61) == 0           # few rows are taken as they are
    assert ws(0, 32, 61, AL, 61, AL, 64) == 0
    ws = capi.sgemm_i8_grouped_workspace
    assert ws(2, 64, 32, 64, AL, 64, AL, 64, 2048) == 0
    assert ws(2, 64, 32, 64, AL, 64, AL, 64, 2049) == 2 * 32 * 64
    assert ws(1, 64, 32, 64, AL, 64, AL, 64, 2049) == 0         # one group has no stride
    ws = capi.sgemm_grouped_sort_workspace
    assert ws(1024, 2, 4096) == 0 and ws(-1, 2, 3) == DIM and ws(5, 5, 5000) == DIM
    for T, picks, groups in ((2049, 1, 3), (16384, 8, 128), (1 << 27, 8, 4096)):
        assert 0 < ws(T, picks, groups) <= 4 * (1 << 17)


def _meta(shape, dtype, strides=None):
    import torch
    t = torch.empty(0, dtype=dtype, device="meta")
    if strides is None:
        strides = [1] * len(shape)
        for i in range(len(shape) - 2, -1, -1):
            strides[i] = strides[i + 1] * shape[i + 1]
    return t.as_strided(shape, strides)


def test_python_refusals_without_a_device():
    import torch

    import fp32_sgemm_tuning_amd as lib
    i8, f32, bf, i32 = torch.int8, torch.float32, torch.bfloat16, torch.int32

    def m(rows, K, **kw):
        return lib.I8Matrix(torch.zeros(rows, K, dtype=kw.get("values", i8)), torch.ones(kw.get("n", rows), dtype=kw.get("scales", f32)))
    wrong = {
        TypeError: [lambda: lib.sgemm_i8(m(2, 8, values=torch.uint8), m(3, 8)), lambda: lib.sgemm_i8(m(2, 8), m(3, 8, scales=bf)),
                    lambda: lib.sgemm_i8_quantize(torch.zeros(2, 3, dtype=torch.float64)), lambda: lib.sgemm_i8_dequantize(m(2, 3), torch.int32),
                    lambda: lib.sgemm_grouped_sort(torch.zeros(4, 8), torch.zeros(4, 2), 3), lambda: lib.sgemm_grouped_sort(torch.zeros(4, 8, dtype=i8), torch.zeros(4, 2, dtype=i32), 3)],
        ValueError: [lambda: lib.sgemm_i8(m(2, 8), m(3, 9)), lambda: lib.sgemm_i8(m(2, 8, n=3), m(3, 8)), lambda: lib.sgemm_i8(m(2, 8), m(3, 8)),
                     lambda: lib.sgemm_i8(lib.I8Matrix(torch.zeros(8, 2, dtype=i8).T, torch.ones(2)), m(3, 8)),
                     lambda: lib.sgemm_i8_grouped(m(2, 8), m(3, 8), torch.zeros(2, dtype=i32)),
                     lambda: lib.sgemm_i8_quantize(torch.zeros(5)), lambda: lib.sgemm_i8_quantize(torch.zeros(5, 4)),
                     lambda: lib.sgemm_grouped_sort(torch.zeros(3, 8), torch.zeros(4, 2, dtype=i32), 3),
                     lambda: lib.sgemm_grouped_sort(torch.zeros(4, 8), torch.zeros(4, 2, 1, dtype=i32), 3),
                     lambda: lib.sgemm_grouped_sort(torch.zeros(4, 8), torch.zeros(2, 4, dtype=i32).T, 3),
                     lambda: lib.sgemm_grouped_sort(torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32), -1),
                     lambda: lib.sgemm_grouped_sort(torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32), 3)]}
    order = lib.GroupOrder(torch.zeros(4, dtype=i32), torch.zeros(4, 2, dtype=i32), torch.zeros(8, dtype=i32))
    Y = torch.zeros(8, 16)
    wrong[TypeError] += [lambda: lib.sgemm_grouped_combine(Y, order._replace(position=order.position.long())),
                         lambda: lib.sgemm_grouped_combine(Y.to(bf), order, out_dtype=torch.float16), lambda: lib.sgemm_grouped_combine(Y.int(), order),
                         lambda: lib.sgemm_grouped_combine(Y, order, torch.zeros(4, 2, dtype=torch.float64)),
                         lambda: lib.sgemm_grouped_combine_grad(torch.zeros(4, 16, dtype=bf), Y.to(torch.float16), order)]
    wrong[ValueError] += [lambda: lib.sgemm_grouped_combine(Y[:7], order), lambda: lib.sgemm_grouped_combine(Y, order, torch.zeros(2, 4)),
                          lambda: lib.sgemm_grouped_combine(Y, order._replace(source=order.source[:7])), lambda: lib.sgemm_grouped_combine(Y, order),
                          lambda: lib.sgemm_grouped_combine(Y, order._replace(position=torch.zeros(2, 4, dtype=i32).T)),
                          lambda: lib.sgemm_grouped_combine_grad(torch.zeros(4, 15), Y, order)]
    for error, calls in wrong.items():
        for i, call in enumerate(calls):
            with pytest.raises(error):
                call()
                pytest.fail(f"{error.__name__} {i}")


def test_sizes_past_an_int_are_refused():
    import torch

    import fp32_sgemm_tuning_amd as lib
    far, i8 = 2 ** 32 + 64, torch.int8

    def m(rows, K, ld):
        return lib.I8Matrix(_meta((rows, K), i8, (ld, 1)), _meta((rows,), torch.float32))
    e, order = _meta((4, 2), torch.int64), lib.GroupOrder(_meta((4,), torch.int32), _meta((4, 2), torch.int32), _meta((8,), torch.int32))
    calls = [lambda: lib.sgemm_i8(m(4, 64, far), m(4, 64, 64)), lambda: lib.sgemm_i8(m(4, 64, 64), m(far, 64, 64)),
             lambda: lib.sgemm_i8_grouped(m(4, 64, far), lib.I8Matrix(_meta((1, 4, 64), i8), _meta((1, 4), torch.float32)), _meta((2,), torch.int32)),
             lambda: lib.sgemm_i8_quantize(_meta((4, 8), torch.float32, (far, 1))), lambda: lib.sgemm_i8_quantize(_meta((3, 2 ** 30, 8), torch.float32)),
             lambda: lib.sgemm_i8_dequantize(m(4, 64, far)),
             lambda: lib.sgemm_grouped_sort(_meta((4, 8), torch.float32, (far, 1)), e, 3), lambda: lib.sgemm_grouped_sort(None, _meta((4, 2), torch.int64, (far, 1)), 3),
             lambda: lib.sgemm_grouped_sort(None, _meta((2 ** 30, 2), torch.int64), 3), lambda: lib.sgemm_grouped_sort(None, e, far),
             lambda: lib.sgemm_grouped_combine(_meta((8, 8), torch.float32, (far, 1)), order),
             lambda: lib.sgemm_grouped_combine(_meta((8, 8), torch.float32), order, _meta((4, 2), torch.float32, (far, 1))),
             lambda: lib.sgemm_grouped_combine_grad(_meta((4, 8), torch.float32, (far, 1)), _meta((8, 8), torch.float32), order)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()
            pytest.fail(str(i))


def test_first_call_of_a_process(monkeypatch):
    """A result's type code is known before any call has looked one up."""
    import torch

    import fp32_sgemm_tuning_amd as lib
    monkeypatch.setattr(lib, "_CODES", {})
    assert lib._result(None, (2, 3), None, torch.zeros(1))[1:] == (capi.SGEMM_DTYPE_F32, 3)
    monkeypatch.setattr(lib, "_CODES", {})
    assert lib._result(torch.zeros(2, 3, dtype=torch.bfloat16), (2, 3), None, None)[1:] == (capi.SGEMM_DTYPE_BF16, 3)


def test_scales_of_rows_without_columns_need_their_source():
    """Rows of no columns may be NULL; their scales, if wanted, are still read from somewhere."""
    args = dict(SORT, dtype=4, H=0, X=None, rows=None, row_scales=AL)
    assert capi.sgemm_grouped_sort(**args) == NULL


def test_rows_of_groups_too_far_apart():
    """Groups of one row: the step between the groups is the rows', the unused step of a group's only row is not looked at."""
    import torch

    import fp32_sgemm_tuning_amd as lib
    with pytest.raises(ValueError, match="below 2\\^31"):
        lib.sgemm_i8_quantize(_meta((3, 1, 8), torch.float32, (2 ** 31, 8, 1)))
    with pytest.raises(ValueError, match="below 2\\^31"):
        lib.sgemm_i8_dequantize(lib.I8Matrix(_meta((3, 1, 8), torch.int8, (2 ** 31, 8, 1)), _meta((3, 1), torch.float32)))
    with pytest.raises(ValueError, match="device tensors"):
        lib.sgemm_i8_quantize(_meta((3, 1, 8), torch.float32, (8, 2 ** 31, 1)))

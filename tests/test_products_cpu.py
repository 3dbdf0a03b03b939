"""Argument checks of the grouped products, the output layer with its loss
and the 4-bit weights: every call below returns before any HIP call."""
import pytest

from fp32_sgemm_tuning_amd import capi

AL, MIS = 0x10000, 0x10002          # fake device addresses, aligned and not; never dereferenced

GROUPED = dict(dtype=1, op_b=0, groups=2, M=64, N=32, K=16, alpha=1.0, A=AL, lda=16, B=AL, ldb=32, stride_b=512,
               offsets=AL, beta=0.0, C=AL, ldc=32, dtype_c=3, workspace=None, workspace_bytes=0, stream=None)
WGRAD = dict(dtype=2, groups=2, M=64, N=32, K=16, alpha=1.0, A=AL, lda=16, D=AL, ldd=32, offsets=AL, beta=0.0, C=AL,
             ldc=32, stride_c=512, dtype_c=2, workspace=None, workspace_bytes=0, stream=None)
XENT = dict(dtype=1, M=8, N=100, K=16, alpha=1.0, X=AL, ldx=16, W=AL, ldw=16, target=AL, ignore_index=-100, loss=AL,
            lse=AL, workspace=AL, workspace_bytes=1 << 40, stream=None)
GRAD = dict(dtype=1, M=8, N=100, K=16, alpha=1.0, X=AL, ldx=16, W=AL, ldw=16, target=AL, ignore_index=-100, lse=AL,
            dloss=AL, dloss_stride=1, dX=AL, lddx=16, dW=AL, lddw=16, workspace=AL, workspace_bytes=1 << 40,
            stream=None)
W4 = dict(dtype=1, M=3, N=32, K=128, alpha=1.0, X=AL, ldx=128, packed=AL, scales=AL, zeros=None, group=128, beta=0.0,
          C=AL, ldc=32, dtype_c=1, workspace=None, workspace_bytes=0, stream=None)
PACK = dict(dtype=1, N=32, K=128, W=AL, ldw=128, group=64, packed=AL, scales=AL, zeros=None, stream=None)
UNPACK = dict(dtype=1, N=32, K=128, packed=AL, scales=AL, zeros=None, group=64, W=AL, ldw=128, stream=None)

DIM, NULL, OP, TYPE, SMALL, UNSUP = (capi.SGEMM_STATUS_INVALID_DIM, capi.SGEMM_STATUS_NULL_POINTER,
                                     capi.SGEMM_STATUS_INVALID_OP, capi.SGEMM_STATUS_INVALID_DTYPE,
                                     capi.SGEMM_STATUS_SCRATCH_TOO_SMALL, capi.SGEMM_STATUS_UNSUPPORTED)

REFUSED = [
    (capi.sgemm_lowp_grouped, GROUPED, [
        (TYPE, dict(dtype=3)), (TYPE, dict(dtype=0)), (TYPE, dict(dtype_c=2)), (OP, dict(op_b=2)),
        (DIM, dict(M=-1)), (DIM, dict(N=-1)), (DIM, dict(K=-1)), (DIM, dict(groups=-1)), (DIM, dict(groups=65536)),
        (DIM, dict(lda=15)), (DIM, dict(ldb=31)), (DIM, dict(ldc=31)), (DIM, dict(op_b=1, ldb=15)),
        (DIM, dict(stride_b=-1)), (DIM, dict(N=1 << 23, ldb=1 << 23, ldc=1 << 23)),
        (DIM, dict(M=2 ** 31 - 1, N=1 << 21, ldb=1 << 21, ldc=1 << 21)),
        (NULL, dict(A=None)), (NULL, dict(B=None)), (NULL, dict(C=None)), (NULL, dict(offsets=None)),
        (SMALL, dict(lda=17)), (SMALL, dict(A=MIS)), (SMALL, dict(stride_b=513)),
        (SMALL, dict(A=MIS, workspace=AL, workspace_bytes=64 * 16 * 2 - 1)),
        (SMALL, dict(A=MIS, workspace=MIS, workspace_bytes=1 << 30))]),
    (capi.sgemm_lowp_grouped_wgrad, WGRAD, [
        (TYPE, dict(dtype=3)), (TYPE, dict(dtype_c=1)), (DIM, dict(M=-1)), (DIM, dict(groups=65536)),
        (DIM, dict(lda=15)), (DIM, dict(ldd=31)), (DIM, dict(ldc=31)), (DIM, dict(stride_c=511)),
        (DIM, dict(groups=60000, K=1 << 20, N=1 << 20, lda=1 << 20, ldd=1 << 20, ldc=1 << 20, stride_c=1 << 40)),
        (NULL, dict(A=None)), (NULL, dict(D=None)), (NULL, dict(C=None)), (NULL, dict(offsets=None)),
        (SMALL, dict(ldd=33)), (SMALL, dict(K=15)), (SMALL, dict(M=4000)),
        (SMALL, dict(M=4000, workspace=AL, workspace_bytes=7 * 2 * 16 * 32 * 4 - 1))]),
    (capi.sgemm_lowp_xent, XENT, [
        (TYPE, dict(dtype=3)), (DIM, dict(M=-1)), (DIM, dict(N=0)), (DIM, dict(K=-1)), (DIM, dict(ldx=15)),
        (DIM, dict(ldw=15)), (DIM, dict(M=(1 << 24) + 1)), (DIM, dict(N=(1 << 30) + 1)),
        (NULL, dict(X=None)), (NULL, dict(W=None)), (NULL, dict(target=None)), (NULL, dict(loss=None)), (NULL, dict(lse=None)), (SMALL, dict(workspace=None)),
        (SMALL, dict(workspace=MIS)), (SMALL, dict(workspace_bytes=100))]),
    (capi.sgemm_lowp_xent_grad, GRAD, [
        (TYPE, dict(dtype=3)), (DIM, dict(M=-1)), (DIM, dict(N=0)), (DIM, dict(ldx=15)), (DIM, dict(lddx=15)),
        (DIM, dict(lddw=15)), (DIM, dict(dloss_stride=-1)), (NULL, dict(X=None)), (NULL, dict(W=None)),
        (NULL, dict(target=None)), (NULL, dict(lse=None)), (NULL, dict(dloss=None)), (SMALL, dict(workspace=None)),
        (SMALL, dict(workspace_bytes=100))]),
    (capi.sgemm_w4, W4, [
        (TYPE, dict(dtype=3)), (TYPE, dict(dtype_c=2)), (DIM, dict(M=-1)), (DIM, dict(N=-1)), (DIM, dict(K=-1)),
        (DIM, dict(group=16)), (DIM, dict(group=256)), (DIM, dict(ldx=127)), (DIM, dict(ldc=31)),
        (NULL, dict(X=None)), (NULL, dict(packed=None)), (NULL, dict(scales=None)), (NULL, dict(C=None)),
        (UNSUP, dict(packed=0x10008)), (UNSUP, dict(scales=0x10004)), (UNSUP, dict(zeros=0x10002)),
        (DIM, dict(M=(1 << 24) + 1)), (DIM, dict(K=1 << 23, ldx=1 << 23)),
        (DIM, dict(M=1 << 24, N=1 << 30, ldc=1 << 30)), (SMALL, dict(X=MIS)),
        (SMALL, dict(ldx=129, workspace=AL, workspace_bytes=3 * 256 - 1))]),
    (capi.sgemm_w4_quantize, PACK, [
        (TYPE, dict(dtype=3)), (DIM, dict(N=-1)), (DIM, dict(group=48)), (DIM, dict(ldw=127)), (NULL, dict(W=None)),
        (NULL, dict(packed=None)), (NULL, dict(scales=None)), (UNSUP, dict(packed=0x10004))]),
    (capi.sgemm_w4_dequantize, UNPACK, [
        (TYPE, dict(dtype=0)), (DIM, dict(K=-1)), (DIM, dict(group=0)), (DIM, dict(ldw=127)), (NULL, dict(W=None)),
        (NULL, dict(packed=None)), (NULL, dict(scales=None)), (UNSUP, dict(packed=0x10004))]),
]


@pytest.mark.parametrize("call,good,want,bad", [(c, g, w, b) for c, g, cases in REFUSED for w, b in cases],
                         ids=lambda v: getattr(v, "__name__", None) or (str(v)[:40] if isinstance(v, dict) and len(v) < 8 else ""))
def test_refused(call, good, want, bad):
    assert call(**{**good, **bad}) == want


@pytest.mark.parametrize("call,good,empty", [
    (capi.sgemm_lowp_grouped, GROUPED, dict(M=0)), (capi.sgemm_lowp_grouped, GROUPED, dict(N=0)),
    (capi.sgemm_lowp_grouped, GROUPED, dict(groups=0)), (capi.sgemm_lowp_grouped_wgrad, WGRAD, dict(groups=0)),
    (capi.sgemm_lowp_grouped_wgrad, WGRAD, dict(N=0, stride_c=0)), (capi.sgemm_lowp_xent, XENT, dict(M=0)),
    (capi.sgemm_lowp_xent_grad, GRAD, dict(dX=None, dW=None)), (capi.sgemm_lowp_xent_grad, GRAD, dict(K=0)),
    (capi.sgemm_w4, W4, dict(M=0)), (capi.sgemm_w4, W4, dict(N=0)), (capi.sgemm_w4_quantize, PACK, dict(N=0)),
    (capi.sgemm_w4_dequantize, UNPACK, dict(K=0))])
def test_empty_calls_launch_nothing(call, good, empty):
    assert call(**{**good, **empty}) == capi.SGEMM_STATUS_OK


def test_workspaces():
    """None for operands taken as they are, else the zero-padded copies."""
    ws = capi.sgemm_lowp_grouped_workspace
    assert ws(0, 2, 64, 32, 16, AL, 16, AL, 32, 512) == 0
    assert ws(0, 2, 64, 32, 16, AL, 17, AL, 32, 512) == 64 * 16 * 2
    assert ws(0, 2, 64, 32, 13, AL, 13, AL, 32, 512) == 64 * 16 * 2           # rows of B past K are not read
    assert ws(1, 2, 64, 30, 13, AL, 13, AL, 13, 390) == 64 * 16 * 2 + 2 * 30 * 16 * 2
    assert ws(2, 2, 64, 32, 16, AL, 16, AL, 32, 512) == OP
    assert capi.sgemm_lowp_grouped_wgrad_workspace(2, 64, 32, 16, AL, 16, AL, 32) == 0
    assert capi.sgemm_lowp_grouped_wgrad_workspace(2, 64, 30, 16, AL, 16, AL, 30) == 64 * 32 * 2
    # 4000 rows of 2 groups: seven shares of 256 rows or more
    assert capi.sgemm_lowp_grouped_wgrad_workspace(2, 4000, 32, 16, AL, 16, AL, 32) == 7 * 2 * 16 * 32 * 4
    assert capi.sgemm_lowp_grouped_wgrad_workspace(2, 4000, 4096, 4096, AL, 4096, AL, 4096) == 0
    assert capi.sgemm_lowp_xent_workspace(0, 100, 16, AL, 16, AL, 16, 0) == 0
    # the backward keeps one piece of the vocabulary: far less than the logits
    M, N, K = 8192, 128000, 4096
    assert capi.sgemm_lowp_xent_workspace(M, N, K, AL, K, AL, K, 1) < M * N * 2 // 4
    assert capi.sgemm_lowp_xent_workspace(M, N, K, AL, K, AL, K, 0) < M * N * 2 // 8


    assert capi.sgemm_w4_workspace(3, 128, AL, 128) == 0
    assert capi.sgemm_w4_workspace(3, 125, AL, 128) == 3 * 128 * 2


def test_python_refusals_without_a_device():
    import torch

    import fp32_sgemm_tuning_amd as lib
    e = torch.bfloat16
    x = torch.ones(4, 8, dtype=e)
    with pytest.raises(ValueError):
        lib.sgemm_grouped(x, torch.ones(1, 8, 8, dtype=e), torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError):
        lib.sgemm_xent(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        lib.sgemm_w4_quantize(x)
    with pytest.raises(TypeError):
        lib.sgemm_w4_quantize(x.float())
    with pytest.raises(ValueError):
        lib.sgemm_w4(x, lib.W4Weight(torch.zeros(4, 64, dtype=torch.uint8), torch.ones(4, 1, dtype=e), None, 8, 48))

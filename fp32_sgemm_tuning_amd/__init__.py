"""MI355X-native FP32 SGEMM (C = alpha*A*B + beta*C, row-major) for gfx950.

The GEMM runs in hand-written HIP kernels in ``libsgemm.so`` (C ABI in
include/sgemm.h, raw binding in :mod:`.capi`).  This module marshals torch
tensors into that call: device pointers, leading dimensions and the current
HIP stream.  PyTorch only supplies device memory and streams.
"""
import contextlib
from typing import NamedTuple, Optional

from . import capi

__all__ = ["sgemm", "sgemm_op", "sgemm_lowp", "sgemm_grouped", "sgemm_grouped_wgrad", "sgemm_xent", "sgemm_xent_grad",
           "sgemm_w4", "sgemm_w4_quantize", "sgemm_w4_dequantize", "W4Weight", "SgemmError", "capi", "variant_names"]


class SgemmError(RuntimeError):
    def __init__(self, status: int):
        msg = capi.sgemm_strerror(status)
        if status == capi.SGEMM_STATUS_HIP_ERROR:
            msg += ": " + capi.sgemm_last_hip_error()
        super().__init__(f"sgemm failed with status {status}: {msg}")
        self.status = status


def _ld(t, name, dtypes=None):
    import torch
    if t.dtype not in (dtypes or (torch.float32,)):
        raise TypeError(f"{name} must be " + " or ".join(str(d).replace("torch.", "") for d in (dtypes or (torch.float32,))))
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    # A single row (or an empty matrix) has no meaningful row stride; keep a
    # padded view's stride when it is valid, else use the packed one.
    if rows > 1 or t.stride(0) >= max(cols, 1):
        return t.stride(0)
    return max(cols, 1)


def sgemm(A, B, C=None, alpha=1.0, beta=0.0, variant=None, stream=None):
    """C = alpha * A @ B + beta * C on the current device; returns C.

    A [M,K], B [K,N], C [M,N] are float32 CUDA/HIP tensors with unit column
    stride (padded rows are fine).  With C None a new tensor is allocated
    (then beta must be 0).  ``variant`` forces a kernel variant (tests and
    sweeps); ``stream`` is a torch stream (default: the current stream).
    """
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C has shape {tuple(C.shape)}, expected {(M, N)}")
    lda, ldb, ldc = _ld(A, "A"), _ld(B, "B"), _ld(C, "C")
    _same_device(A, B, C)
    with _device_ctx(A.device):
        args = (M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
                float(beta), C.data_ptr(), ldc, _stream_handle(A.device, stream))
        if variant is None:
            st = capi.sgemm(*args)
        else:
            st = capi.sgemm_ex(*args, int(variant))
    if st != capi.SGEMM_STATUS_OK:
        raise SgemmError(st)
    return C


def _same_device(A, B, C):
    if not (A.device == B.device == C.device):
        raise ValueError(f"A, B and C must be on one device, got {A.device}, {B.device}, {C.device}")


def _device_ctx(device):
    """A context with `device` current; nothing to do when it already is."""
    import torch
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_handle(device, stream):
    """The HIP stream handle of `stream` (a torch stream), else of the
    device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    idx = device.index if device.index is not None else torch.cuda.current_device()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(idx)
    return torch.cuda.current_stream(idx).cuda_stream


def variant_names():
    return [capi.sgemm_variant_name(v) for v in range(capi.sgemm_num_variants())]


def _mat(t, name, dtypes=None):
    """(rows, cols, ld) of a row-major matrix view, or of each matrix of a
    3-D batch view (then also the batch stride)."""
    import torch
    if t.dtype not in (dtypes or (torch.float32,)):
        raise TypeError(f"{name} has type {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() == 2:
        return t.shape[0], t.shape[1], _ld(t, name, dtypes), 0
    if t.dim() == 3:
        rows, cols = t.shape[1], t.shape[2]
        if cols > 1 and t.stride(2) != 1:
            raise ValueError(f"{name} must have unit column stride (row-major)")
        ld = t.stride(1) if rows > 1 or t.stride(1) >= max(cols, 1) else max(cols, 1)
        return rows, cols, ld, t.stride(0) if t.shape[0] > 1 else 0
    raise ValueError(f"{name} must be 2-D or 3-D")


def sgemm_op(A, B, C=None, alpha=1.0, beta=0.0, trans_a=False, trans_b=False, stream=None):
    """C = alpha * op(A) @ op(B) + beta * C with op(X) = X or X^T, row-major;
    returns C.

    A and B are the stored matrices: with trans_a, A is [K,M]; with trans_b,
    B is [N,K].  3-D tensors ([batch, rows, cols], any batch stride, one of A
    and B may have batch 1 to be shared) run as one strided batch.
    """
    import torch
    batched = A.dim() == 3 or B.dim() == 3 or (C is not None and C.dim() == 3)
    ra, ca, lda, sa = _mat(A, "A")
    rb, cb, ldb, sb = _mat(B, "B")
    M, K = (ca, ra) if trans_a else (ra, ca)
    K2, N = (cb, rb) if trans_b else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: op(A) is {M}x{K}, op(B) is {K2}x{N}")
    batch = max(A.shape[0] if A.dim() == 3 else 1, B.shape[0] if B.dim() == 3 else 1)
    for t, name in ((A, "A"), (B, "B")):
        if t.dim() == 3 and t.shape[0] not in (1, batch):
            raise ValueError(f"{name} has batch {t.shape[0]}, expected 1 or {batch}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((batch, M, N) if batched else (M, N), dtype=torch.float32, device=A.device)
    rc, cc, ldc, sc = _mat(C, "C")
    _same_device(A, B, C)
    if (rc, cc) != (M, N) or (C.dim() == 3 and C.shape[0] != batch):
        raise ValueError(f"C has shape {tuple(C.shape)}, expected {(batch, M, N) if batched else (M, N)}")
    op_a = capi.SGEMM_OP_T if trans_a else capi.SGEMM_OP_N
    op_b = capi.SGEMM_OP_T if trans_b else capi.SGEMM_OP_N
    with _device_ctx(A.device):
        h = _stream_handle(A.device, stream)
        if batched:
            st = capi.sgemm_strided_batched(op_a, op_b, M, N, K, float(alpha), A.data_ptr(), lda, sa,
                                            B.data_ptr(), ldb, sb, float(beta), C.data_ptr(), ldc, sc, batch, h)
        else:
            st = capi.sgemm_op(op_a, op_b, M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
                               float(beta), C.data_ptr(), ldc, h)
    if st != capi.SGEMM_STATUS_OK:
        raise SgemmError(st)
    return C


def sgemm_lowp(A, B, C=None, alpha=1.0, beta=0.0, variant=None, stream=None, trans_a=False, trans_b=False):
    """C = alpha * op(A) @ op(B) + beta * C with bfloat16 or float16 A and B
    (one type for both, unit column stride) and FP32 accumulation; C is
    float32 (allocated when None, then beta must be 0); returns C.  op(X) =
    X, or X^T with trans_a / trans_b (then A is stored [K,M], B [N,K]).  3-D
    tensors ([batch, rows, cols], any batch stride, one of A and B may have
    batch 1 to be shared) run as one strided batch.  ``variant`` forces a
    kernel variant of a single untransposed problem (tests and sweeps)."""
    import torch
    codes = {torch.bfloat16: capi.SGEMM_DTYPE_BF16, torch.float16: capi.SGEMM_DTYPE_F16}
    batched = A.dim() == 3 or B.dim() == 3 or (C is not None and C.dim() == 3)
    ra, ca, lda, sa = _mat(A, "A", tuple(codes))
    rb, cb, ldb, sb = _mat(B, "B", tuple(codes))
    if B.dtype != A.dtype:
        raise TypeError(f"A is {A.dtype} but B is {B.dtype}")
    M, K = (ca, ra) if trans_a else (ra, ca)
    K2, N = (cb, rb) if trans_b else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: op(A) is {M}x{K}, op(B) is {K2}x{N}")
    batch = max(A.shape[0] if A.dim() == 3 else 1, B.shape[0] if B.dim() == 3 else 1)
    for t, name in ((A, "A"), (B, "B")):
        if t.dim() == 3 and t.shape[0] not in (1, batch):
            raise ValueError(f"{name} has batch {t.shape[0]}, expected 1 or {batch}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((batch, M, N) if batched else (M, N), dtype=torch.float32, device=A.device)
    rc, cc, ldc, sc = _mat(C, "C")
    if (rc, cc) != (M, N) or (C.dim() == 3 and C.shape[0] != batch):
        raise ValueError(f"C has shape {tuple(C.shape)}, expected {(batch, M, N) if batched else (M, N)}")
    _same_device(A, B, C)
    op_a = capi.SGEMM_OP_T if trans_a else capi.SGEMM_OP_N
    op_b = capi.SGEMM_OP_T if trans_b else capi.SGEMM_OP_N
    with _device_ctx(A.device):
        h = _stream_handle(A.device, stream)
        if batched:
            st = capi.sgemm_lowp_strided_batched(codes[A.dtype], op_a, op_b, M, N, K, float(alpha), A.data_ptr(),
                                                 lda, sa, B.data_ptr(), ldb, sb, float(beta), C.data_ptr(), ldc, sc,
                                                 batch, h)
        elif trans_a or trans_b:
            st = capi.sgemm_lowp_op(codes[A.dtype], op_a, op_b, M, N, K, float(alpha), A.data_ptr(), lda,
                                    B.data_ptr(), ldb, float(beta), C.data_ptr(), ldc, h,
                                    capi.SGEMM_VARIANT_AUTO if variant is None else int(variant))
        else:
            args = (codes[A.dtype], M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
                    float(beta), C.data_ptr(), ldc, h)
            st = capi.sgemm_lowp(*args) if variant is None else capi.sgemm_lowp_ex(*args, int(variant))
    if st != capi.SGEMM_STATUS_OK:
        raise SgemmError(st)
    return C


# ---------------------------------------------------------------------------
# Products grouped by rows, the output layer with its loss, 4-bit weights.
# ---------------------------------------------------------------------------
_CODES = {}     # torch type -> element type code


def _codes():
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: capi.SGEMM_DTYPE_BF16, torch.float16: capi.SGEMM_DTYPE_F16,
                       torch.float32: capi.SGEMM_DTYPE_F32})
    return _CODES


def _inputs16():
    import torch
    return torch.bfloat16, torch.float16


def _one_device(*named):
    """The device of the (name, tensor) pairs (None tensors left out); an error if they are on several."""
    device = named[0][1].device
    for name, t in named:
        if t is not None and t.device != device:
            raise ValueError("operands must be on one device, got " +
                             ", ".join(f"{n} on {x.device}" for n, x in named if x is not None))
    if device.type != "cuda":
        raise ValueError("operands must be device tensors")
    return device


def _vector(t, name, dtype, size):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.dim() != 1 or t.shape[0] != size:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(size,)}")
    if size > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


class _On:
    """`device` current, and `stream` (if given) current on it, so that what
    is allocated for a call belongs to the stream the call runs on; gives the
    stream's handle."""
    __slots__ = ("device", "stream", "stack")

    def __init__(self, device, stream):
        self.device, self.stream, self.stack = device, stream, None

    def __enter__(self):
        import torch
        inner = _device_ctx(self.device)
        if self.stream is not None or not isinstance(inner, contextlib.nullcontext):
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(inner)
            if self.stream is not None:
                self.stack.enter_context(torch.cuda.stream(self.stream))
        return _stream_handle(self.device, self.stream)

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()


def _check(status):
    if status < 0:
        raise SgemmError(status)
    return status


def _with_workspace(call, size, device):
    """call(workspace address, bytes), with a workspace of size() bytes if it
    asks for one (it has then enqueued nothing)."""
    status = call(None, 0)
    if status == capi.SGEMM_STATUS_SCRATCH_TOO_SMALL:
        import torch
        n = _check(size())
        keep = torch.empty(n, dtype=torch.uint8, device=device)
        status = call(keep.data_ptr(), n)
    _check(status)


def _result(C, shape, out_dtype, default, allowed, beta, device):
    """The result tensor of a call, checked or allocated."""
    import torch
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty(shape, dtype=out_dtype or default, device=device)
    elif out_dtype is not None and C.dtype != out_dtype:
        raise TypeError(f"C is {C.dtype} but out_dtype is {out_dtype}")
    if C.dtype not in allowed:
        raise TypeError(f"C has type {C.dtype}")
    if tuple(C.shape) != tuple(shape):
        raise ValueError(f"C has shape {tuple(C.shape)}, expected {tuple(shape)}")
    return C


def _offsets(offsets):
    import torch
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be int32")
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must hold groups + 1 row numbers")
    if offsets.shape[0] > 1 and offsets.stride(0) != 1:
        raise ValueError("offsets must be contiguous")
    return offsets.shape[0] - 1


def sgemm_grouped(A, B, offsets, C=None, alpha=1.0, beta=0.0, trans_b=False, out_dtype=None, stream=None):
    """C[r] = alpha * A[r] @ op(B[g]) + beta * C[r] for the rows r of each
    group g, offsets[g] <= r < offsets[g+1]; returns C.

    A [T,K] bfloat16 or float16, B [G,K,N] (with trans_b [G,N,K]) of the same
    type, offsets int32 [G+1] on the device, not decreasing, within 0..T.
    C [T,N] is float32 (the default) or of A's type (out_dtype).  Groups may
    be empty; rows of no group are left as they were (uninitialised in a C
    allocated here).  The gradient with respect to A is this call on dC with
    trans_b turned round; with respect to B see sgemm_grouped_wgrad."""
    import torch
    groups = _offsets(offsets)
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be 2-D and B 3-D")
    M, K, lda, _ = _mat(A, "A", _inputs16())
    rb, cb, ldb, sb = _mat(B, "B", _inputs16())
    if B.dtype != A.dtype:
        raise TypeError(f"A is {A.dtype} but B is {B.dtype}")
    K2, N = (cb, rb) if trans_b else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A is {M}x{K}, op(B[g]) is {K2}x{N}")
    if B.shape[0] != groups:
        raise ValueError(f"B holds {B.shape[0]} matrices, offsets bound {groups} groups")
    device = _one_device(("A", A), ("B", B), ("offsets", offsets), ("C", C))
    with _On(device, stream) as h:
        C = _result(C, (M, N), out_dtype, torch.float32, (torch.float32, A.dtype), beta, device)
        ldc = _ld(C, "C", (C.dtype,))
        op = capi.SGEMM_OP_T if trans_b else capi.SGEMM_OP_N
        b_args = (A.data_ptr(), lda, B.data_ptr(), ldb, sb)
        args = (_codes()[A.dtype], op, groups, M, N, K, float(alpha), *b_args, offsets.data_ptr(), float(beta),
                C.data_ptr(), ldc, _codes()[C.dtype])
        _with_workspace(lambda ws, size: capi.sgemm_lowp_grouped(*args, ws, size, h),
                        lambda: capi.sgemm_lowp_grouped_workspace(op, groups, M, N, K, *b_args), device)
    return C


def sgemm_grouped_wgrad(A, D, offsets, C=None, alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """C[g] = alpha * A[r].T @ D[r] + beta * C[g] over the rows r of each
    group g (as in sgemm_grouped); returns C [G,K,N].

    A [T,K] and D [T,N] bfloat16 or float16; C float32 (the default) or of
    A's type.  An empty group gives beta * C[g].  With C = A @ B[g] per group,
    dB = sgemm_grouped_wgrad(A, dC, offsets); for weights stored [G,N,K]
    (trans_b) the operands change places."""
    import torch
    groups = _offsets(offsets)
    M, K, lda, _ = _mat(A, "A", _inputs16())
    M2, N, ldd, _ = _mat(D, "D", _inputs16())
    if A.dim() != 2 or D.dim() != 2:
        raise ValueError("A and D must be 2-D")
    if D.dtype != A.dtype:
        raise TypeError(f"A is {A.dtype} but D is {D.dtype}")
    if M2 != M:
        raise ValueError(f"A has {M} rows, D has {M2}")
    device = _one_device(("A", A), ("D", D), ("offsets", offsets), ("C", C))
    with _On(device, stream) as h:
        C = _result(C, (groups, K, N), out_dtype, torch.float32, (torch.float32, A.dtype), beta, device)
        _, _, ldc, sc = _mat(C, "C", (C.dtype,))
        a_args = (A.data_ptr(), lda, D.data_ptr(), ldd)
        args = (_codes()[A.dtype], groups, M, N, K, float(alpha), *a_args, offsets.data_ptr(), float(beta),
                C.data_ptr(), ldc, sc, _codes()[C.dtype])
        _with_workspace(lambda ws, size: capi.sgemm_lowp_grouped_wgrad(*args, ws, size, h),
                        lambda: capi.sgemm_lowp_grouped_wgrad_workspace(M, N, K, *a_args), device)
    return C


def _xent_args(X, W, target):
    import torch
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and W must be 2-D")
    M, K, ldx, _ = _mat(X, "X", _inputs16())
    N, K2, ldw, _ = _mat(W, "W", _inputs16())
    if W.dtype != X.dtype:
        raise TypeError(f"X is {X.dtype} but W is {W.dtype}")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {N}x{K2}")
    if N < 1:
        raise ValueError("W holds no rows")
    _vector(target, "target", torch.int64, M)
    return M, N, K, ldx, ldw


def sgemm_xent(X, W, target, alpha=1.0, ignore_index=-100, stream=None):
    """(loss, lse), float32 [T] each, of the logits l = alpha * X @ W.T:
    lse = log(sum(exp(l))), loss = lse - l[target], without the logits being
    kept.

    X [T,H] and W [V,H] bfloat16 or float16, target int64 [T].  Rows whose
    target is ignore_index give 0 in both; any other target outside 0..V-1
    gives a NaN loss."""
    import torch
    M, N, K, ldx, ldw = _xent_args(X, W, target)
    device = _one_device(("X", X), ("W", W), ("target", target))
    with _On(device, stream) as h:
        loss = torch.empty(M, dtype=torch.float32, device=device)
        lse = torch.empty(M, dtype=torch.float32, device=device)
        args = (X.data_ptr(), ldx, W.data_ptr(), ldw)
        size = _check(capi.sgemm_lowp_xent_workspace(M, N, K, *args, 0))
        keep = torch.empty(size, dtype=torch.uint8, device=device)
        _check(capi.sgemm_lowp_xent(_codes()[X.dtype], M, N, K, float(alpha), *args, target.data_ptr(),
                                    int(ignore_index), loss.data_ptr(), lse.data_ptr(), keep.data_ptr(), size, h))
    return loss, lse


def sgemm_xent_grad(X, W, target, lse, dloss, alpha=1.0, ignore_index=-100, need_dx=True, need_dw=True, stream=None):
    """(dX, dW), the gradients of sum(dloss * loss) for the loss and lse of
    sgemm_xent on the same arguments; of X's type.

    dloss float32 [T], or one value ([] or [1]) for all rows.  need_dx /
    need_dw False: None in that place, and no work for it (a frozen W)."""
    import torch
    M, N, K, ldx, ldw = _xent_args(X, W, target)
    _vector(lse, "lse", torch.float32, M)
    if dloss.dtype != torch.float32:
        raise TypeError("dloss must be float32")
    if dloss.numel() == 1:
        step = 0
    elif dloss.dim() == 1 and dloss.shape[0] == M and dloss.stride(0) >= 0:
        step = dloss.stride(0)
    else:
        raise ValueError(f"dloss has shape {tuple(dloss.shape)}, expected {(M,)} or one value")
    device = _one_device(("X", X), ("W", W), ("target", target), ("lse", lse), ("dloss", dloss))
    with _On(device, stream) as h:
        dX = torch.empty((M, K), dtype=X.dtype, device=device) if need_dx else None
        dW = torch.empty((N, K), dtype=X.dtype, device=device) if need_dw else None
        args = (X.data_ptr(), ldx, W.data_ptr(), ldw)
        size = _check(capi.sgemm_lowp_xent_workspace(M, N, K, *args, 1))
        keep = torch.empty(size, dtype=torch.uint8, device=device)
        _check(capi.sgemm_lowp_xent_grad(_codes()[X.dtype], M, N, K, float(alpha), *args, target.data_ptr(),
                                         int(ignore_index), lse.data_ptr(), dloss.data_ptr(), step,
                                         dX.data_ptr() if need_dx else None, max(K, 1),
                                         dW.data_ptr() if need_dw else None, max(K, 1), keep.data_ptr(), size, h))
    return dX, dW


class W4Weight(NamedTuple):
    """A weight [N,K] in 4 bits, w = (q - z) * s with a scale s and a zero
    point z for each `group` (32, 64 or 128) consecutive k of a row.

    With Kp = K rounded up to 128: packed uint8 [N, Kp/2] (16-byte aligned;
    64 bytes hold 128 k as 32-bit words, word 4j + s of them k = 32s + 8j..+7,
    element 2i in bits 4i..4i+3, element 2i+1 in bits 16+4i..16+4i+3), scales
    [N, Kp/group] of the inputs' type (8-byte aligned), zeros uint8
    [N, Kp/group] with values 0..15 (4-byte aligned), or None (every z is 8);
    all contiguous."""
    packed: "torch.Tensor"              # noqa: F821
    scales: "torch.Tensor"              # noqa: F821
    zeros: "Optional[torch.Tensor]"     # noqa: F821
    K: int
    group: int


def _w4(W):
    """(N, checked) of a W4Weight."""
    import torch
    if W.group not in (32, 64, 128):
        raise ValueError(f"group is {W.group}, expected 32, 64 or 128")
    if W.packed.dtype != torch.uint8 or W.packed.dim() != 2:
        raise TypeError("packed must be a uint8 matrix")
    if W.scales.dtype not in _inputs16():
        raise TypeError(f"scales has type {W.scales.dtype}")
    N, Kp = W.packed.shape[0], (W.K + 127) // 128 * 128
    if W.zeros is not None and W.zeros.dtype != torch.uint8:
        raise TypeError("zeros must be uint8")
    for t, name, cols in ((W.packed, "packed", Kp // 2), (W.scales, "scales", Kp // W.group),
                          (W.zeros, "zeros", Kp // W.group)):
        if t is not None and (tuple(t.shape) != (N, cols) or not t.is_contiguous()):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected contiguous {(N, cols)}")
    return N


def _address(t):
    return None if t is None else t.data_ptr()


def sgemm_w4(X, W, C=None, alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """C = alpha * X @ W.T + beta * C for a 4-bit weight W (W4Weight [N,K]);
    returns C.

    X [M,K] bfloat16 or float16, any M from a single token to a prompt; the
    scales are of X's type.  C [M,N] is float32 (the default) or of X's
    type."""
    import torch
    N = _w4(W)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K, ldx, _ = _mat(X, "X", _inputs16())
    if W.scales.dtype != X.dtype:
        raise TypeError(f"X is {X.dtype} but the scales are {W.scales.dtype}")
    if K != W.K:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {N}x{W.K}")
    device = _one_device(("X", X), ("packed", W.packed), ("scales", W.scales), ("zeros", W.zeros), ("C", C))
    with _On(device, stream) as h:
        C = _result(C, (M, N), out_dtype, torch.float32, (torch.float32, X.dtype), beta, device)
        ldc = _ld(C, "C", (C.dtype,))
        x, codes = X.data_ptr(), _codes()
        args = (codes[X.dtype], M, N, K, float(alpha), x, ldx, W.packed.data_ptr(), W.scales.data_ptr(),
                _address(W.zeros), W.group, float(beta), C.data_ptr(), ldc, codes[C.dtype])
        _with_workspace(lambda ws, size: capi.sgemm_w4(*args, ws, size, h),
                        lambda: capi.sgemm_w4_workspace(M, K, x, ldx), device)
    return C


def sgemm_w4_quantize(W, group=128, zeros=False, stream=None):
    """W [N,K] (bfloat16 or float16) as a W4Weight: one scale per `group`
    consecutive k, and with `zeros` a zero point (for groups that lie to one
    side of 0)."""
    import torch
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    N, K, ldw, _ = _mat(W, "W", _inputs16())
    if group not in (32, 64, 128):
        raise ValueError(f"group is {group}, expected 32, 64 or 128")
    Kp = (K + 127) // 128 * 128
    device = _one_device(("W", W))
    with _On(device, stream) as h:
        out = W4Weight(torch.empty((N, Kp // 2), dtype=torch.uint8, device=device),
                       torch.empty((N, Kp // group), dtype=W.dtype, device=device),
                       torch.empty((N, Kp // group), dtype=torch.uint8, device=device) if zeros else None, K, group)
        _check(capi.sgemm_w4_quantize(_codes()[W.dtype], N, K, W.data_ptr(), ldw, group, out.packed.data_ptr(),
                                      out.scales.data_ptr(), _address(out.zeros), h))
    return out


def sgemm_w4_dequantize(W, stream=None):
    """The values [N,K] a W4Weight stands for, rounded to its scales' type."""
    import torch
    N = _w4(W)
    device = _one_device(("packed", W.packed), ("scales", W.scales), ("zeros", W.zeros))
    with _On(device, stream) as h:
        out = torch.empty((N, W.K), dtype=W.scales.dtype, device=device)
        _check(capi.sgemm_w4_dequantize(_codes()[out.dtype], N, W.K, W.packed.data_ptr(), W.scales.data_ptr(),
                                        _address(W.zeros), W.group, out.data_ptr(), max(W.K, 1), h))
    return out

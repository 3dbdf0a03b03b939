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


_INT = 2 ** 31 - 1   # sizes and leading dimensions are C ints; ctypes would drop higher bits unseen


def _too_large(name):
    raise ValueError(f"{name}: sizes and row strides must be below 2^31")


def _rows16(t, name):
    """(type code, rows, columns, leading dimension) of a 16-bit row-major matrix view."""
    code = _codes().get(t.dtype, 0)
    if code not in (capi.SGEMM_DTYPE_BF16, capi.SGEMM_DTYPE_F16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    step, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    # (a single row, or none, has no meaningful row stride)
    ld = step if rows > 1 or step >= cols > 0 else max(cols, 1)
    if rows | cols | ld > _INT:
        _too_large(name)
    return code, rows, cols, ld


def _same_type(a, a_name, b, b_name):
    if a.dtype != b.dtype:
        raise TypeError(f"{a_name} is {a.dtype} but {b_name} is {b.dtype}")


def _one_device(first, *named):
    """The index of the device of `first` and of the (name, tensor) pairs (None tensors left out)."""
    index = first.get_device()
    if index < 0:
        raise ValueError("operands must be device tensors")
    for name, t in named:
        if t is not None and t.get_device() != index:
            raise ValueError(f"operands must be on one device: {name} is on {t.device}, not on {first.device}")
    return index


def _vector(t, name, dtype, size):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.dim() != 1 or t.shape[0] != size:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(size,)}")
    if size > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _run(index, stream, call, *operands):
    """call(stream handle), with the device current and `stream` (if given)
    current on it, so that what it allocates belongs to the stream it runs on;
    the operands' memory is then kept until that stream has used it."""
    import torch
    if stream is None and index == torch.cuda.current_device():
        return call(_stream_handle(operands[0].device, None))
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream belongs to {stream.device}, the operands to {operands[0].device}")
    with torch.cuda.device(index), (torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()):
        if stream is not None:
            for t in operands:
                if t is not None:
                    t.record_stream(stream)
        return call(_stream_handle(operands[0].device, stream))


def _check(status):
    if status < 0:
        raise SgemmError(status)
    return status


def _finish(status, call, size, operand):
    """After call(None, 0) gave `status`: an error, or again with a workspace
    of size() bytes if it asks for one (it has then enqueued nothing)."""
    if status == capi.SGEMM_STATUS_SCRATCH_TOO_SMALL:
        import torch
        n = _check(size())
        keep = operand.new_empty(n, dtype=torch.uint8)
        status = call(keep.data_ptr(), n)
    _check(status)


def _check_result(C, shape, out_dtype, operand, beta):
    """Before anything is allocated: beta, a given C's shape and type, the wanted type."""
    import torch
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        if out_dtype is not None and out_dtype not in (torch.float32, operand.dtype):
            raise TypeError(f"out_dtype is {out_dtype}, expected float32 or {operand.dtype}")
        return
    if out_dtype is not None and C.dtype != out_dtype:
        raise TypeError(f"C is {C.dtype} but out_dtype is {out_dtype}")
    if C.dtype not in (torch.float32, operand.dtype):
        raise TypeError(f"C has type {C.dtype}, expected float32 or {operand.dtype}")
    if tuple(C.shape) != shape:
        raise ValueError(f"C has shape {tuple(C.shape)}, expected {shape}")
    if shape[-1] > 1 and C.stride(-1) != 1:
        raise ValueError("C must have unit column stride (row-major)")


def _result(C, shape, out_dtype, operand):
    """(C, its type's code, leading dimension), allocated here where it is None."""
    import torch
    rows, cols = shape[-2:]
    if C is None:
        dtype = out_dtype or torch.float32
        return operand.new_empty(shape, dtype=dtype), _CODES[dtype], max(cols, 1)
    step = C.stride(-2)
    ld = step if rows > 1 or step >= cols > 0 else max(cols, 1)
    if ld > _INT:
        _too_large("C")
    return C, _CODES[C.dtype], ld


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
    groups = _offsets(offsets)
    code, M, K, lda = _rows16(A, "A")
    if B.dim() != 3:
        raise ValueError("B must be 3-D")
    _same_type(A, "A", B, "B")
    held, rb, cb = B.shape
    sb, ldb, unit = B.stride()
    if unit != 1 and cb > 1:
        raise ValueError("B must have unit column stride (row-major)")
    ldb = ldb if rb > 1 or ldb >= cb > 0 else max(cb, 1)
    if held | rb | cb | ldb > _INT:
        _too_large("B")
    K2, N = (cb, rb) if trans_b else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A is {M}x{K}, op(B[g]) is {K2}x{N}")
    if held != groups:
        raise ValueError(f"B holds {held} matrices, offsets bound {groups} groups")
    device = _one_device(A, ("B", B), ("offsets", offsets), ("C", C))
    _check_result(C, (M, N), out_dtype, A, beta)
    op = capi.SGEMM_OP_T if trans_b else capi.SGEMM_OP_N
    operands = (A.data_ptr(), lda, B.data_ptr(), ldb, sb if held > 1 else 0)

    def call(h):
        out, code_c, ldc = _result(C, (M, N), out_dtype, A)
        args = (code, op, groups, M, N, K, float(alpha), *operands, offsets.data_ptr(), float(beta), out.data_ptr(),
                ldc, code_c)
        product = capi.load().sgemm_lowp_grouped
        status = product(*args, None, 0, h)
        if status:
            _finish(status, lambda ws, size: product(*args, ws, size, h),
                    lambda: capi.sgemm_lowp_grouped_workspace(op, groups, M, N, K, *operands), A)
        return out
    return _run(device, stream, call, A, B, offsets, C)


def sgemm_grouped_wgrad(A, D, offsets, C=None, alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """C[g] = alpha * A[r].T @ D[r] + beta * C[g] over the rows r of each
    group g (as in sgemm_grouped); returns C [G,K,N].

    A [T,K] and D [T,N] bfloat16 or float16; C float32 (the default) or of
    A's type.  An empty group gives beta * C[g].  With C = A @ B[g] per group,
    dB = sgemm_grouped_wgrad(A, dC, offsets); for weights stored [G,N,K]
    (trans_b) the operands change places."""
    groups = _offsets(offsets)
    code, M, K, lda = _rows16(A, "A")
    _, M2, N, ldd = _rows16(D, "D")
    _same_type(A, "A", D, "D")
    if M2 != M:
        raise ValueError(f"A has {M} rows, D has {M2}")
    device = _one_device(A, ("D", D), ("offsets", offsets), ("C", C))
    _check_result(C, (groups, K, N), out_dtype, A, beta)
    operands = (A.data_ptr(), lda, D.data_ptr(), ldd)

    def call(h):
        out, code_c, ldc = _result(C, (groups, K, N), out_dtype, A)
        args = (code, groups, M, N, K, float(alpha), *operands, offsets.data_ptr(), float(beta), out.data_ptr(), ldc,
                out.stride(0) if groups > 1 else 0, code_c)
        product = capi.load().sgemm_lowp_grouped_wgrad
        status = product(*args, None, 0, h)
        if status:
            _finish(status, lambda ws, size: product(*args, ws, size, h),
                    lambda: capi.sgemm_lowp_grouped_wgrad_workspace(groups, M, N, K, *operands), A)
        return out
    return _run(device, stream, call, A, D, offsets, C)


def _xent_args(X, W, target):
    import torch
    code, M, K, ldx = _rows16(X, "X")
    _, N, K2, ldw = _rows16(W, "W")
    _same_type(X, "X", W, "W")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {N}x{K2}")
    if N < 1:
        raise ValueError("W holds no rows")
    _vector(target, "target", torch.int64, M)
    return code, M, N, K, (X.data_ptr(), ldx, W.data_ptr(), ldw)


def sgemm_xent(X, W, target, alpha=1.0, ignore_index=-100, stream=None):
    """(loss, lse), float32 [T] each, of the logits l = alpha * X @ W.T:
    lse = log(sum(exp(l))), loss = lse - l[target], without the logits being
    kept.

    X [T,H] and W [V,H] bfloat16 or float16, target int64 [T].  Rows whose
    target is ignore_index give 0 in both; any other target outside 0..V-1
    gives a NaN loss."""
    import torch
    code, M, N, K, operands = _xent_args(X, W, target)
    device = _one_device(X, ("W", W), ("target", target))
    size = _check(capi.sgemm_lowp_xent_workspace(M, N, K, *operands, 0))

    def call(h):
        loss, lse = X.new_empty(M, dtype=torch.float32), X.new_empty(M, dtype=torch.float32)
        ws = X.new_empty(size, dtype=torch.uint8)
        _check(capi.sgemm_lowp_xent(code, M, N, K, float(alpha), *operands, target.data_ptr(), int(ignore_index), loss.data_ptr(),
                                    lse.data_ptr(), ws.data_ptr(), size, h))
        return loss, lse
    return _run(device, stream, call, X, W, target)


def sgemm_xent_grad(X, W, target, lse, dloss, alpha=1.0, ignore_index=-100, need_dx=True, need_dw=True, stream=None):
    """(dX, dW), the gradients of sum(dloss * loss) for the loss and lse of
    sgemm_xent on the same arguments; of X's type.

    dloss float32 [T], or one value ([] or [1]) for all rows.  need_dx /
    need_dw False: None in that place, and no work for it (a frozen W)."""
    import torch
    code, M, N, K, operands = _xent_args(X, W, target)
    _vector(lse, "lse", torch.float32, M)
    if dloss.dtype != torch.float32:
        raise TypeError("dloss must be float32")
    if dloss.numel() == 1 and dloss.dim() <= 1:
        step = 0
    elif dloss.dim() == 1 and dloss.shape[0] == M:
        step = dloss.stride(0)
        if step > _INT:
            _too_large("dloss")
    else:
        raise ValueError(f"dloss has shape {tuple(dloss.shape)}, expected {(M,)} or one value")
    device = _one_device(X, ("W", W), ("target", target), ("lse", lse), ("dloss", dloss))
    size = _check(capi.sgemm_lowp_xent_workspace(M, N, K, *operands, 1))

    def call(h):
        dX = X.new_empty((M, K)) if need_dx else None
        dW = X.new_empty((N, K)) if need_dw else None
        ws = X.new_empty(size, dtype=torch.uint8)
        _check(capi.sgemm_lowp_xent_grad(code, M, N, K, float(alpha), *operands, target.data_ptr(), int(ignore_index),
                                         lse.data_ptr(), dloss.data_ptr(), step, _address(dX), max(K, 1), _address(dW),
                                         max(K, 1), ws.data_ptr(), size, h))
        return dX, dW
    return _run(device, stream, call, X, W, target, lse, dloss)


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
    """The rows of a W4Weight, its parts checked."""
    import torch
    packed, scales, zeros, K, group = W
    if group not in (32, 64, 128):
        raise ValueError(f"group is {group}, expected 32, 64 or 128")
    if packed.dtype != torch.uint8 or packed.dim() != 2:
        raise TypeError("packed must be a uint8 matrix")
    if scales.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"scales has type {scales.dtype}")
    if zeros is not None and zeros.dtype != torch.uint8:
        raise TypeError("zeros must be uint8")
    N, Kp = packed.shape[0], (K + 127) // 128 * 128
    if N | K > _INT:
        _too_large("weight")
    if packed.shape[1] != Kp // 2 or not packed.is_contiguous():
        raise ValueError(f"packed has shape {tuple(packed.shape)}, expected contiguous {(N, Kp // 2)}")
    for t, name in ((scales, "scales"), (zeros, "zeros")):
        if t is not None and (t.shape != (N, Kp // group) or not t.is_contiguous()):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected contiguous {(N, Kp // group)}")
    return N


def _address(t):
    return None if t is None else t.data_ptr()


def sgemm_w4(X, W, C=None, alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """C = alpha * X @ W.T + beta * C for a 4-bit weight W (W4Weight [N,K]);
    returns C.

    X [M,K] bfloat16 or float16, any M from a single token to a prompt; the
    scales are of X's type.  C [M,N] is float32 (the default) or of X's
    type."""
    N = _w4(W)
    code, M, K, ldx = _rows16(X, "X")
    packed, scales, zeros, WK, group = W
    _same_type(X, "X", scales, "scales")
    if K != WK:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {N}x{WK}")
    device = _one_device(X, ("packed", packed), ("scales", scales), ("zeros", zeros), ("C", C))
    _check_result(C, (M, N), out_dtype, X, beta)

    def call(h):
        out, code_c, ldc = _result(C, (M, N), out_dtype, X)
        x = X.data_ptr()
        args = (code, M, N, K, float(alpha), x, ldx, packed.data_ptr(), scales.data_ptr(), _address(zeros), group,
                float(beta), out.data_ptr(), ldc, code_c)
        product = capi.load().sgemm_w4
        status = product(*args, None, 0, h)
        if status:
            _finish(status, lambda ws, size: product(*args, ws, size, h), lambda: capi.sgemm_w4_workspace(M, K, x, ldx), X)
        return out
    return _run(device, stream, call, X, packed, scales, zeros, C)


def sgemm_w4_quantize(W, group=128, zeros=False, stream=None):
    """W [N,K] (bfloat16 or float16) as a W4Weight: one scale per `group`
    consecutive k, and with `zeros` a zero point (for groups that lie to one
    side of 0)."""
    import torch
    code, N, K, ldw = _rows16(W, "W")
    if group not in (32, 64, 128):
        raise ValueError(f"group is {group}, expected 32, 64 or 128")
    Kp = (K + 127) // 128 * 128
    device = _one_device(W)

    def call(h):
        out = W4Weight(W.new_empty((N, Kp // 2), dtype=torch.uint8), W.new_empty((N, Kp // group)),
                       W.new_empty((N, Kp // group), dtype=torch.uint8) if zeros else None, K, group)
        _check(capi.sgemm_w4_quantize(code, N, K, W.data_ptr(), ldw, group, out.packed.data_ptr(),
                                      out.scales.data_ptr(), _address(out.zeros), h))
        return out
    return _run(device, stream, call, W)


def sgemm_w4_dequantize(W, stream=None):
    """The values [N,K] a W4Weight stands for, rounded to its scales' type."""
    N = _w4(W)
    packed, scales, zeros, K, group = W
    device = _one_device(packed, ("scales", scales), ("zeros", zeros))

    def call(h):
        out = scales.new_empty((N, K))
        _check(capi.sgemm_w4_dequantize(_codes()[out.dtype], N, K, packed.data_ptr(), scales.data_ptr(),
                                        _address(zeros), group, out.data_ptr(), max(K, 1), h))
        return out
    return _run(device, stream, call, packed, scales, zeros)

/*
 * sgemm.h - C ABI of the MI355X (gfx950) single-precision GEMM library
 * (libsgemm.so).
 *
 * Operation.  C = alpha * A * B + beta * C for row-major FP32 matrices
 * A [M,K], B [K,N] and C [M,N]; each output is a length-K dot product and the
 * whole product counts 2*M*N*K FLOPs ("Matmul I: tiling and shared memory",
 * section 1).  The epilogue has the form alpha*acc + beta*C ("2D Register
 * Tiling: The Outer Product", The Kernel) and, when beta == 0, C is never
 * read ("The Final Kernel: Retuning Against the Pipeline", Skipping The Read
 * Of C), so NaN or Inf already in C cannot reach the result.  Elements outside
 * the matrices contribute nothing and only in-range outputs are written
 * ("Matmul I", section 6).
 *
 * Layout.  Element (i,k) of A is A[i*lda + k], (k,j) of B is B[k*ldb + j],
 * (i,j) of C is C[i*ldc + j]; lda >= max(1,K), ldb >= max(1,N),
 * ldc >= max(1,N).  Columns j in [N, ldc) of C are never written.
 * Arithmetic is FP32 (v_mfma_f32_16x16x4_f32 matrix instructions, FP32
 * accumulate); no reduced-precision inputs are used.
 *
 * Pointers.  A, B and C are device pointers of the current HIP device.
 * C must not overlap A or B (not checked).  Any alignment is accepted: when
 * A, B and C are 16-byte aligned and lda, ldb, ldc are multiples of 4 the
 * library uses 128-bit loads and stores, otherwise 32-bit ones.
 *
 * Ownership and execution.  The caller owns A, B and C.  A call validates
 * its arguments, enqueues one kernel on `stream` (a hipStream_t; NULL is the
 * null stream; two kernels when the last wave of tiles is split, see
 * sgemm_tail_split) and returns without synchronising.  Calls are thread-safe
 * and deterministic: the same inputs and the same split of K (see
 * "Workspace") give the same bits.
 *
 * Workspace.  Small tile grids split K over several workgroups per output
 * tile (split-K).  Those calls use a workspace of SGEMM_WORKSPACE_BYTES
 * (64 MiB of partial tiles and 4096 tile counters) that the library
 * allocates with hipMalloc for a stream on its first such call.  A device
 * keeps at most SGEMM_MAX_STREAM_WORKSPACES of them, each bound to one stream
 * (the per-thread default stream counts once per host thread); when more
 * streams ask, the least recently used workspace that no call in progress
 * holds is handed to the new stream once the kernels queued on it have
 * finished, so device memory stays bounded however many streams a process
 * creates and destroys.  Until a stream first finds every workspace of its
 * device taken, calls record nothing at their end (each stream keeps its
 * workspace); that call waits once for the device to drain
 * (hipDeviceSynchronize) before it takes over an idle workspace, and from
 * then on every split call records an event at its end that marks the
 * workspace's last use.  The counters are cleared on the stream before a workspace's
 * first use and left cleared by every call.  Calls on one stream share its
 * workspace in stream order.  The partial tiles of a tile are added in a
 * fixed order, so split-K results are deterministic too.  A call that finds
 * no workspace free without waiting for another call (every one held at
 * that moment), and every call on a stream under graph capture, runs with K
 * unsplit: the same result within rounding, nothing allocated or waited
 * for.  No call waits while holding the library's lock, so calls on
 * different streams never block each other.  An allocation failure returns
 * SGEMM_STATUS_HIP_ERROR before anything is enqueued.  sgemm_op(), sgemm_cm()
 * and sgemm_lowp() keep copy buffers the same way (see sgemm_op).
 * sgemm_workspace_bytes() reports the device memory held and
 * sgemm_release_workspaces() frees it.
 *
 * HIP errors.  Every launch's status is taken from the launch call itself:
 * the library never calls hipGetLastError or hipPeekAtLastError, so it
 * neither consumes a HIP error the caller left pending nor reports such an
 * error as its own.
 *
 * Errors.  Arguments are checked before anything is enqueued, so a call that
 * returns an error has written nothing.  M == 0 or N == 0 returns
 * SGEMM_STATUS_OK without launching.  K == 0 writes alpha*0 + beta*C
 * (alpha*0 when beta == 0).
 */
#ifndef SGEMM_MI355X_H
#define SGEMM_MI355X_H

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_STATUS_OK 0
#define SGEMM_STATUS_INVALID_DIM (-1)       /* M, N, K < 0, or a leading dimension too small, or too many tiles */
#define SGEMM_STATUS_NULL_POINTER (-2)      /* NULL A, B or C with a non-empty extent */
#define SGEMM_STATUS_HIP_ERROR (-3)         /* the HIP runtime reported an error; see sgemm_last_hip_error() */
#define SGEMM_STATUS_INVALID_VARIANT (-4)   /* sgemm_ex: no such variant */
#define SGEMM_STATUS_UNSUPPORTED (-5)       /* a forced variant, or a packed weight, needs 16-byte alignment */
#define SGEMM_STATUS_INVALID_OP (-6)        /* an operation code other than SGEMM_OP_N / SGEMM_OP_T */

#define SGEMM_STATUS_INVALID_DTYPE (-7)     /* an element type the call does not take */
#define SGEMM_STATUS_SCRATCH_TOO_SMALL (-8) /* the call needs more scratch or workspace than it has */

/* Device memory the library keeps between calls (see "Workspace" above). */
#define SGEMM_WORKSPACE_BYTES (64ll * 1024 * 1024 + 16 * 1024)  /* one split-K workspace */
#define SGEMM_MAX_STREAM_WORKSPACES 8       /* split-K workspaces kept per device */
#define SGEMM_MAX_COPY_BUFFERS 2            /* copy buffers kept per device */
#define SGEMM_MAX_COPY_BUFFER_BYTES (4ll << 30)  /* largest copy buffer; larger copies are not made */
#define SGEMM_NOALLOC_SCRATCH_BYTES (64ll * 1024 * 1024 + 16 * 1024)  /* sgemm_noalloc's static scratch, per device */

/* Element types of sgemm_lowp and the calls below it. */
#define SGEMM_DTYPE_BF16 1                  /* bfloat16: 1 sign, 8 exponent, 7 fraction bits */
#define SGEMM_DTYPE_F16 2                   /* IEEE binary16 */
#define SGEMM_DTYPE_F32 3                   /* IEEE binary32: result type of the grouped, 4-bit and 8-bit products */
#define SGEMM_DTYPE_I8 4                    /* 8-bit integers with a scale for each row: rows that sgemm_grouped_sort takes */

/* Operation codes of the sgemm_op family. */
#define SGEMM_OP_N 0                        /* use the stored matrix as is */
#define SGEMM_OP_T 1                        /* use the transpose of the stored matrix */

/* Variant ids for sgemm_ex(). */
#define SGEMM_VARIANT_AUTO (-1)             /* what sgemm() picks */
#define SGEMM_VARIANT_SIMPLE 0              /* 64x64 tile, single LDS buffer, 32-bit loads: the plain cross-check kernel */
#define SGEMM_VARIANT_DB128_VEC 1           /* 128x128x32 tile, double-buffered LDS, 128-bit loads/stores (needs alignment) */
#define SGEMM_VARIANT_DB128_SCALAR 2        /* the same tile with 32-bit loads/stores (any alignment) */
/* Ids 3 .. sgemm_num_variants()-1 are further kernels and tile shapes with
 * 128-bit access (double-buffered, section-pipelined, direct-to-LDS, lean
 * direct-to-LDS, and the split-K form of the lean 128x128x32 kernel), kept
 * for tile sweeps; sgemm_variant_name() and sgemm_variant_info() describe
 * them.  The direct-to-LDS kernels take the shapes they support (whole tiles,
 * or for the lean kernels K >= the K tile with K and N multiples of 4) and
 * use the guarded kernel of the same tile otherwise. */

/*
 * sgemm: C = alpha*A*B + beta*C (see above).  Picks the kernel variant from
 * the alignment class and the shape: the lean direct-to-LDS kernel with
 * 16-byte loads when the operands allow 128-bit access, else with 4-byte
 * loads (any alignment); on 64x64x64 block tiles when a 128x128 grid would
 * have at most 256 tiles or a less full last wave over the 256 compute
 * units, else on 128x128x32 tiles.  The 64x64x64 forms split K when their
 * own grid is under one wave of resident blocks (512 tiles) and splitting
 * saves time by the library's cost model (see sgemm_split_factor), and
 * split the last wave of a larger grid (see sgemm_tail_split).  Shapes a
 * lean kernel does not take go to a guarded kernel.  beta == 0 selects an
 * epilogue that never reads C.  Returns SGEMM_STATUS_*.
 */
int sgemm(int M, int N, int K, float alpha,
          const float *A, int lda,
          const float *B, int ldb,
          float beta, float *C, int ldc,
          void *stream);

/*
 * sgemm_ex: as sgemm() with the kernel variant forced (SGEMM_VARIANT_*; AUTO
 * behaves like sgemm()).  Intended for tests and tile sweeps.  Returns
 * SGEMM_STATUS_INVALID_VARIANT for an unknown id and SGEMM_STATUS_UNSUPPORTED
 * when a 128-bit variant is forced on arguments that lack its alignment.
 */
int sgemm_ex(int M, int N, int K, float alpha,
             const float *A, int lda,
             const float *B, int ldb,
             float beta, float *C, int ldc,
             void *stream, int variant);

/*
 * sgemm_noalloc: sgemm() for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc).  Same arguments, operation, variant choice and split of K as
 * sgemm(), so the same bits; it never calls hipMalloc or hipFree, on the
 * first call or later.  Its split-K partial tiles and tile counters live in
 * a static device array of SGEMM_NOALLOC_SCRATCH_BYTES that the library's
 * code holds on every device it is loaded on, until the process ends; the
 * first call on a device looks up that array's address there.  Each call
 * that splits K first clears the counters it uses with a small kernel on
 * `stream` (no memset, so the call can be captured into a graph; under
 * capture K is split as outside it).  Every call on a device shares that
 * device's array and the array keeps the last call's contents: calls that
 * overlap in time on one device (on different streams, or from different
 * host threads) race and must be ordered by the caller; calls in order on
 * one stream are safe.  The array holds 64 MiB of partial tiles, as much
 * as a split-K workspace, and sgemm() keeps every split within that (the
 * automatic choice reaches 63 MiB on large 128x128 grids whose last wave
 * splits; SGEMM_SPLITK is clamped to it), so every plan fits;
 * SGEMM_STATUS_SCRATCH_TOO_SMALL, with nothing enqueued, guards a plan that
 * would not.  Other statuses as for sgemm().
 */
int sgemm_noalloc(int M, int N, int K, float alpha,
                  const float *A, int lda,
                  const float *B, int ldb,
                  float beta, float *C, int ldc,
                  void *stream);

/*
 * sgemm_select_variant: the variant id sgemm() would run for these arguments
 * (no launch, no HIP call; pointers are only inspected for alignment).
 * Returns a negative status for invalid arguments.
 */
int sgemm_select_variant(int M, int N, int K,
                         const float *A, int lda,
                         const float *B, int ldb,
                         float beta, const float *C, int ldc);

/* Number of variant ids (valid ids are 0 .. n-1). */
int sgemm_num_variants(void);

/* Static name of a variant, or NULL for an unknown id. */
const char *sgemm_variant_name(int variant);

/*
 * sgemm_variant_info: block tile (bm x bn, K step bk) of a variant and whether
 * it needs 16-byte aligned operands (needs_vec = 1).  Any output pointer may
 * be NULL.  Returns SGEMM_STATUS_OK or SGEMM_STATUS_INVALID_VARIANT.
 */
int sgemm_variant_info(int variant, int *bm, int *bn, int *bk, int *needs_vec);

/*
 * sgemm_op: C = alpha * op(A) * op(B) + beta * C, row-major, with
 * op(X) = X (SGEMM_OP_N) or X^T (SGEMM_OP_T).  op(A) is M x K and op(B) is
 * K x N: with op_a = SGEMM_OP_T, A is stored K x M (element (i,k) of op(A)
 * at A[k*lda + i], lda >= max(1,M)); with op_b = SGEMM_OP_T, B is stored
 * N x K (element (k,j) of op(B) at B[j*ldb + k], ldb >= max(1,K)).  The
 * untransposed forms have the layout of sgemm().  The operation is the same
 * dot-product definition as sgemm() with the operands read through the
 * transpose ("Matmul I: tiling and shared memory", section 1); the pages
 * stop at packed untransposed operands and name the column-major BLAS
 * convention only in passing.  sgemm_op(N, N, ...) is sgemm().  A
 * transposed operand with 16-byte aligned rows (base, leading dimension and
 * its contiguous extent multiples of 4 floats) is read in its stored
 * orientation with 16-byte loads; such a product on 64x64 tiles splits K
 * (over the whole grid or over its last wave of tiles) by the rule and with
 * the workspaces of sgemm(), so the factor sgemm_split_factor() and
 * sgemm_tail_split() give for the variant lean_64x64x64_w4x1_splitk
 * applies.  One without is, for a problem large
 * enough that the copy takes less time than the product, first transposed
 * into a row-major copy in the stream's copy buffer (allocated with
 * hipMalloc on first need, grown once the kernels queued with it have
 * finished, at most SGEMM_MAX_COPY_BUFFERS per device, handed between
 * streams like the split-K workspaces), and the product then runs as sgemm()
 * on the copy; otherwise, always under graph capture, and when the stream's
 * buffer is held by a call in progress on another host thread, it is
 * gathered with 4-byte loads.  Environment variable SGEMM_PACK = 1 / -1
 * forces the copy on / off, for sweeps.  Returns SGEMM_STATUS_*; SGEMM_STATUS_INVALID_OP for
 * another op code; SGEMM_STATUS_HIP_ERROR if the buffer cannot be allocated
 * (nothing enqueued).
 */
int sgemm_op(int op_a, int op_b, int M, int N, int K, float alpha,
             const float *A, int lda,
             const float *B, int ldb,
             float beta, float *C, int ldc,
             void *stream);

/*
 * sgemm_strided_batched: `batch` independent sgemm_op problems of one shape;
 * problem z uses A + z*stride_a, B + z*stride_b and C + z*stride_c (in
 * elements).  0 <= batch <= 65535.  stride_a and stride_b may be 0 (one
 * operand shared by all problems); the C problems must not overlap:
 * stride_c >= (M-1)*ldc + N when batch > 1.  One kernel launch for the whole
 * batch.  On 64x64 tiles with 16-byte loads K is split as in sgemm() with
 * the tiles of all problems counted together (so a batch of small problems
 * with long K spreads over the chip), using the stream's split-K workspace;
 * other batches do not split.  Unaligned transposed operands are copied as in
 * sgemm_op(), for the whole batch in one launch per operand (an operand of
 * stride 0 once), when the copies' traffic takes less time than the product
 * and the copies fit in SGEMM_MAX_COPY_BUFFER_BYTES; the same buffer rules
 * apply.  batch == 0 is a no-op.  Returns SGEMM_STATUS_*.
 */
int sgemm_strided_batched(int op_a, int op_b, int M, int N, int K, float alpha,
                          const float *A, int lda, long long stride_a,
                          const float *B, int ldb, long long stride_b,
                          float beta, float *C, int ldc, long long stride_c,
                          int batch, void *stream);

/*
 * sgemm_cm, sgemm_cm_strided_batched: the same operations on column-major
 * matrices (the BLAS convention): element (i,j) of an r x c matrix X at
 * X[i + j*ld], ld >= max(1,r); op(A) is M x K, op(B) is K x N, C is M x N
 * with ldc >= max(1,M).  A column-major matrix is the row-major storage of
 * its transpose, so these run the row-major product C^T = op(B)^T op(A)^T.
 */
int sgemm_cm(int op_a, int op_b, int M, int N, int K, float alpha,
             const float *A, int lda,
             const float *B, int ldb,
             float beta, float *C, int ldc,
             void *stream);
int sgemm_cm_strided_batched(int op_a, int op_b, int M, int N, int K, float alpha,
                             const float *A, int lda, long long stride_a,
                             const float *B, int ldb, long long stride_b,
                             float beta, float *C, int ldc, long long stride_c,
                             int batch, void *stream);

/*
 * sgemm_lowp: C = alpha * A * B + beta * C with 16-bit inputs and FP32
 * accumulation and output.  A [M,K] and B [K,N] are row-major arrays of
 * `dtype` elements (SGEMM_DTYPE_BF16 or SGEMM_DTYPE_F16; lda and ldb count
 * elements), C [M,N] is row-major FP32.  The product of two 16-bit values is
 * exact in FP32, so the result is that of sgemm() on the inputs widened to
 * FP32, up to summation order.  The pages name 16-bit inputs on matrix
 * units with FP32 accumulation as the step past FP32 ("gpu_matmul",
 * Conclusion & Next Steps; "The Final Kernel: Retuning Against the
 * Pipeline", What Could Be Improved, And What It Would Take).
 *
 * Fast path: A and B 16-byte aligned, lda, ldb, N and K multiples of 8 and
 * K >= 32.  It runs the matrix instructions v_mfma_f32_16x16x32_bf16 / _f16
 * on 128x128, 256x128 or 256x256 block tiles, picked from the shape, with
 * 16-byte C access when C is 16-byte aligned and ldc a multiple of 4.  Other
 * operands (unaligned rows, K or N not multiples of 8) of a problem with
 * K >= 64, large enough that copying them takes less time than the plain
 * kernel would, are first copied into zero-padded aligned buffers (K and N
 * rounded up to multiples of 8; the stream's copy buffer, as for
 * sgemm_op; an operand the fast path takes as it is, with K a multiple of
 * 8, is used in place) and run on the fast path; the rest (and a call whose stream's
 * buffer is held by another call at that moment) runs a plain kernel that
 * widens each element on load.  SGEMM_PACK = 1 / -1 forces the copy on / off.  Small
 * tile grids split K and use the workspace described above (same rules:
 * allocated on first use per (device, stream), no split under graph
 * capture, deterministic).  Argument checks, layout rules and status codes
 * as for sgemm(), plus SGEMM_STATUS_INVALID_DTYPE, which is checked first.
 */
int sgemm_lowp(int dtype, int M, int N, int K, float alpha,
               const void *A, int lda,
               const void *B, int ldb,
               float beta, float *C, int ldc,
               void *stream);

/*
 * sgemm_lowp_ex: sgemm_lowp() with the kernel variant forced, for tests and
 * tile sweeps: SGEMM_VARIANT_AUTO (-1) behaves like sgemm_lowp(), 0 is the
 * plain kernel (any shape), 1 .. n-1 the matrix-instruction kernel on a block
 * tile and stage count that sgemm_lowp_variant_name() names.  Returns
 * SGEMM_STATUS_INVALID_VARIANT for an unknown id and SGEMM_STATUS_UNSUPPORTED
 * when a variant other than 0 is forced on operands outside its fast path.
 */
int sgemm_lowp_ex(int dtype, int M, int N, int K, float alpha,
                  const void *A, int lda,
                  const void *B, int ldb,
                  float beta, float *C, int ldc,
                  void *stream, int variant);

/*
 * sgemm_lowp_op: sgemm_lowp() with op(A) and op(B) as in sgemm_op(): with
 * op_a = SGEMM_OP_T, A is stored K x M (lda >= max(1,M)); with op_b =
 * SGEMM_OP_T, B is stored N x K (ldb >= max(1,K)); leading dimensions count
 * elements.  `variant` as in sgemm_lowp_ex() (SGEMM_VARIANT_AUTO for the
 * automatic choice); transposed operands run on the alternating-schedule
 * variants or the plain kernel, with each operand kept in LDS in its stored
 * orientation (16-byte chunks along its contiguous extent, which must be a
 * multiple of 8 elements for the fast path).  With transposed operands the
 * 128x128 alternating variant splits K on grids of few tiles, as the
 * 128x128 two-stage kernel does (same workspace
 * rules, deterministic; 512x512x8192 BF16 TN 69 -> 25 us; untransposed
 * operands split on it from 16 tiles up).  With
 * SGEMM_VARIANT_AUTO, operands the fast path cannot take are copied as in
 * sgemm_lowp(), transposed on the way into zero-padded row-major buffers,
 * and the product runs untransposed on the copies (where it may split K,
 * deterministically); an untransposed operand the fast path takes as it is
 * (K a multiple of 8) is used in place.  Returns SGEMM_STATUS_*;
 * SGEMM_STATUS_INVALID_OP for another op code.
 */
int sgemm_lowp_op(int dtype, int op_a, int op_b, int M, int N, int K, float alpha,
                  const void *A, int lda,
                  const void *B, int ldb,
                  float beta, float *C, int ldc,
                  void *stream, int variant);

/*
 * sgemm_lowp_strided_batched: `batch` independent sgemm_lowp_op() problems of
 * one shape, problem z on A + z*stride_a, B + z*stride_b (in 16-bit
 * elements) and C + z*stride_c (in floats); the rules of
 * sgemm_strided_batched() (0 <= batch <= 65535, strides of A and B may be 0,
 * C problems must not overlap, one launch) and the automatic variant choice
 * over batch x tiles; a batch on the 128x128 two-stage kernel or the 128x128
 * alternating kernel splits K over its problems' tiles together
 * (sgemm_lowp_split_factor for untransposed ones).  Batches the fast kernels cannot take
 * (unaligned rows, K or N not multiples of 8, or stride_a or stride_b not a
 * multiple of 8 elements, which leaves problems after the first unaligned)
 * are copied into zero-padded buffers as in sgemm_lowp(), one launch per
 * operand for the whole batch (an operand of stride 0 once), when that
 * takes less time than the plain kernel and the copies fit in
 * SGEMM_MAX_COPY_BUFFER_BYTES; the rest run on the plain kernel.  A
 * transposed batch on the 128x128 alternating kernel splits K as in
 * sgemm_lowp_op(), over its problems' tiles together.  Returns
 * SGEMM_STATUS_*.
 */
int sgemm_lowp_strided_batched(int dtype, int op_a, int op_b, int M, int N, int K, float alpha,
                               const void *A, int lda, long long stride_a,
                               const void *B, int ldb, long long stride_b,
                               float beta, float *C, int ldc, long long stride_c,
                               int batch, void *stream);

/*
 * Products of a language model's weights that a plain product cannot express.
 * All take BF16 or FP16 operands (`dtype`) with FP32 accumulation, run on
 * `stream` without synchronising, keep nothing between calls and allocate
 * nothing: where a call needs device memory of its own the caller passes a
 * 16-byte aligned `workspace` of at least the bytes that the matching
 * *_workspace() function returns for the same arguments (it looks at pointers
 * for their alignment only; 0: pass NULL).  A workspace is free again when
 * the call's work on the stream is done; two calls that may run at the same
 * time, or two captured graphs that may, need one each.  So every call can be
 * captured into a graph.  Results are deterministic.  C must not overlap an
 * operand or the workspace.  Leading dimensions and strides count elements.
 * SGEMM_STATUS_SCRATCH_TOO_SMALL: the workspace is missing, unaligned or too
 * small.  SGEMM_STATUS_INVALID_DIM also where a result has more tiles than one
 * launch covers (2^32 threads): 8.3 million of 256 x 256 outputs in the grouped
 * products (for small groups 16.7 million of 128 x 128 or 32 x 128) and the logits,
 * 8.3 million of 128 x 128 in the weight gradient, 16.7 million of 64 x 128 in the
 * product with 4-bit weights, whose weight may have up to 2^29 - 64 rows.
 *
 * sgemm_lowp_grouped: rows offsets[g] .. offsets[g+1] - 1 of A [M,K] and of
 * C [M,N] belong to group g, whose matrix is op(B) with B at
 * B + g*stride_b, op as in sgemm_lowp_op():
 *   C[rows of g] = alpha * A[rows of g] * op(B[g]) + beta * C[rows of g].
 * `offsets` is a device array of groups + 1 row numbers that do not decrease,
 * within 0 .. M (others are clamped to that range; what an array that
 * decreases leaves in rows of C is unspecified).  Groups may be empty; rows of no group
 * are left as they were.  dtype_c: `dtype` or SGEMM_DTYPE_F32.  The gradient
 * with respect to A is the same call with op_b turned round, the one with
 * respect to B sgemm_lowp_grouped_wgrad.  K and N below 2^22 - 64, groups up
 * to 65535.  Operands whose rows are not whole aligned 16-byte chunks
 * (pointer, leading dimension, row length and stride_b multiples of 8
 * elements) are first copied into zero-padded rows in the workspace.
 */
int sgemm_lowp_grouped(int dtype, int op_b, int groups, int M, int N, int K, float alpha,
                       const void *A, int lda,
                       const void *B, int ldb, long long stride_b,
                       const int *offsets, float beta, void *C, int ldc, int dtype_c,
                       void *workspace, long long workspace_bytes, void *stream);
long long sgemm_lowp_grouped_workspace(int op_b, int groups, int M, int N, int K,
                                       const void *A, int lda,
                                       const void *B, int ldb, long long stride_b);

/*
 * sgemm_lowp_grouped_wgrad: one product per group over the group's rows,
 *   C[g] = alpha * A[rows of g]^T * D[rows of g] + beta * C[g],
 * A [M,K], D [M,N], C[g] K x N at C + g*stride_c (stride_c >=
 * (K-1)*ldc + N when groups > 1).  An empty group gives beta * C[g]
 * (zeros when beta is 0).  Small matrices over many rows are summed in several
 * shares of the rows, whose FP32 products are in the workspace and are added in
 * a fixed order.  Otherwise as sgemm_lowp_grouped().
 */
int sgemm_lowp_grouped_wgrad(int dtype, int groups, int M, int N, int K, float alpha,
                             const void *A, int lda, const void *D, int ldd,
                             const int *offsets, float beta, void *C, int ldc,
                             long long stride_c, int dtype_c,
                             void *workspace, long long workspace_bytes, void *stream);
long long sgemm_lowp_grouped_wgrad_workspace(int groups, int M, int N, int K,
                                             const void *A, int lda,
                                             const void *D, int ldd);

/*
 * sgemm_lowp_xent: the softmax cross entropy of the logits
 * l = alpha * X * W^T, X [M,K] rows, W [N,K] a vocabulary of N >= 1:
 *   lse[i] = log(sum_v exp(l[i][v])),  loss[i] = lse[i] - l[i][target[i]],
 * both FP32, without the M x N logits being in memory.  Rows with
 * target[i] == ignore_index give 0 in both, whatever X holds there; any other
 * target outside 0 .. N-1 gives a NaN loss.  K below 2^22 - 64, M up to 2^24,
 * N up to 2^30.
 */
int sgemm_lowp_xent(int dtype, int M, int N, int K, float alpha,
                    const void *X, int ldx, const void *W, int ldw,
                    const long long *target, long long ignore_index,
                    float *loss, float *lse,
                    void *workspace, long long workspace_bytes, void *stream);

/*
 * sgemm_lowp_xent_grad: the gradients of sum_i dloss[i] * loss[i],
 *   dX = alpha * diag(dloss) * P * W,  dW = alpha * P^T * diag(dloss) * X,
 *   P[i][v] = exp(l[i][v] - lse[i]) - [v == target[i]],
 * with lse from sgemm_lowp_xent() on the same arguments; dX [M,K] and dW
 * [N,K] are of `dtype`, and either may be NULL if it is not wanted.  dloss[i]
 * is at dloss + i*dloss_stride (0: one value for all rows).  Ignored rows
 * give zeros in dX and nothing to dW; rows with a target outside 0 .. N-1
 * (and not ignored) give NaN.  The logits are formed again, a piece of the
 * vocabulary at a time, with P * dloss of that piece in 16 bits in the
 * workspace, scaled so that neither the size of dloss nor (FP16) its spread over
 * the rows costs precision: a term of either sum is off by half a step of
 * `dtype` relative to itself or, if that is more, (FP16) by 2^-34 of its row's
 * |dloss| in dX and 2^-39 of max|dloss| in dW.
 */
int sgemm_lowp_xent_grad(int dtype, int M, int N, int K, float alpha,
                         const void *X, int ldx, const void *W, int ldw,
                         const long long *target, long long ignore_index,
                         const float *lse, const float *dloss, int dloss_stride,
                         void *dX, int lddx, void *dW, int lddw,
                         void *workspace, long long workspace_bytes, void *stream);
long long sgemm_lowp_xent_workspace(int M, int N, int K, const void *X, int ldx,
                                    const void *W, int ldw, int grad);

/*
 * sgemm_w4: C = alpha * X * Wq^T + beta * C, X [M,K] of `dtype`, C [M,N] of
 * `dtype` or SGEMM_DTYPE_F32 (dtype_c), and a weight of 4-bit values,
 *   Wq[n][k] = (q[n][k] - z[n][k / group]) * s[n][k / group],
 * group 32, 64 or 128, the products and sums of unrounded weights in FP32: an
 * infinity or NaN in X gives what this formula does, whatever M, as long as no
 * sum of x * (q - z) over some k of one group passes FP32's range.
 * With Kp = K rounded up to a multiple of 128:
 *   packed  N rows of Kp / 2 bytes, 16-byte aligned, 64 bytes per 128 k: the
 *           32-bit word 4*j + s of a chunk (j, s = 0 .. 3) holds
 *           k = 32*s + 8*j .. + 7 of it, element 2i in bits 4i .. 4i+3 and
 *           element 2i+1 in bits 16+4i .. 16+4i+3
 *   scales  N rows of Kp / group values of `dtype`, 8-byte aligned
 *   zeros   N rows of Kp / group bytes 0 .. 15, 4-byte aligned, or NULL
 *           (every z is 8)
 * What they hold for k >= K, or for a group of such k alone, is not used.
 * SGEMM_STATUS_UNSUPPORTED: one of them is not aligned so.  X whose rows are
 * not whole aligned 16-byte chunks is first copied into the workspace.  M up
 * to 2^24, K below 2^22 - 64.
 */
int sgemm_w4(int dtype, int M, int N, int K, float alpha,
             const void *X, int ldx,
             const void *packed, const void *scales, const void *zeros, int group,
             float beta, void *C, int ldc, int dtype_c,
             void *workspace, long long workspace_bytes, void *stream);
long long sgemm_w4_workspace(int M, int K, const void *X, int ldx);

/* The launch form sgemm_w4() takes for M rows and a weight of N rows (no HIP
 * call): 0, 1, 2 16 rows of X by 16, 32, 64 of W, 3, 4, 5 32 rows by 16, 32, 64,
 * 6, 7 tiles through LDS of 64 x 128, 128 x 128; or SGEMM_STATUS_INVALID_DIM. */
int sgemm_w4_select_form(int M, int N);

/*
 * sgemm_w4_quantize: W [N,K] of `dtype` into the form above (zeros NULL:
 * without zero points).  s is rounded to `dtype` first and q chosen for the
 * rounded s, halves to even:
 *   without  s = max|w| / 7,                       q = round(w / s) + 8
 *   with     s = (max(w, 0) - min(w, 0)) / 15,     z = round(-min(w, 0) / s),
 *            q = round(w / s) + z
 * over the group's k < K, z and q clamped to 0 .. 15; where s is 0, z is 0
 * (with) and q = z.  A group holding a NaN or an infinity gets s NaN.
 * sgemm_w4_dequantize: W = (q - z) * s, rounded to `dtype`.
 */
int sgemm_w4_quantize(int dtype, int N, int K, const void *W, int ldw, int group,
                      void *packed, void *scales, void *zeros, void *stream);
int sgemm_w4_dequantize(int dtype, int N, int K,
                        const void *packed, const void *scales, const void *zeros, int group,
                        void *W, int ldw, void *stream);

/*
 * sgemm_i8: products of 8-bit integers with a scale for each row of X (a
 * token) and each row of W (an output channel),
 *   C[m][n] = alpha * x_scales[m] * w_scales[n] * sum_k X[m][k] * W[n][k]
 *             + beta * C[m][n],
 * X [M,K] and W [N,K] of values -128 .. 127, FP32 scales, C [M,N] of dtype_c:
 * BF16, FP16 or FP32.  The sums are exact (32-bit integers; K up to 131071) and
 * scaled in FP32, (sum * (alpha * x_scales[m])) * w_scales[n], so a result is
 * the same however K is split.  Operands whose rows do not start at multiples of
 * 16 bytes (pointer and leading dimension) are first copied into the workspace
 * (but not for M up to 16 and N up to 2^27 - 16), which also takes the sums of a split
 * K.  An aligned operand is read in whole 16-byte chunks, up to 15 bytes behind the
 * last k of a row; what they hold is not used.  M up to 2^24, N up to 2^30.
 *
 * sgemm_i8_grouped: the same for rows offsets[g] .. offsets[g+1] - 1 of X and of
 * C with the weight at W + g*stride_w and scales at w_scales + g*stride_s;
 * offsets and rows of no group as in sgemm_lowp_grouped(), groups up to 65534,
 * N below 2^22 - 64.  Weights whose rows do not start at multiples of 16 bytes are
 * copied in every call whatever M is, those of empty groups too: lay them out in such
 * rows once.
 */
int sgemm_i8(int M, int N, int K, float alpha,
             const void *X, int ldx, const float *x_scales,
             const void *W, int ldw, const float *w_scales,
             float beta, void *C, int ldc, int dtype_c,
             void *workspace, long long workspace_bytes, void *stream);
long long sgemm_i8_workspace(int M, int N, int K, const void *X, int ldx, const void *W, int ldw);
int sgemm_i8_grouped(int groups, int M, int N, int K, float alpha,
                     const void *X, int ldx, const float *x_scales,
                     const void *W, int ldw, long long stride_w,
                     const float *w_scales, long long stride_s,
                     const int *offsets, float beta, void *C, int ldc, int dtype_c,
                     void *workspace, long long workspace_bytes, void *stream);
long long sgemm_i8_grouped_workspace(int groups, int M, int N, int K, const void *X, int ldx,
                                     const void *W, int ldw, long long stride_w);

/*
 * sgemm_i8_quantize: X [M,K] of BF16, FP16 or FP32 into 8-bit integers with a
 * scale for each row, s = max(max|x| / 127, 2^-126) in FP32 and
 * values = x / s rounded to the nearest integer, halves to even (-127 .. 127).  A
 * row that holds a NaN or an infinity gets s NaN and values 0, so that what is
 * made of it is NaN.  sgemm_i8_dequantize: X = values * s, rounded to `dtype`.  K
 * up to 2^30; M that sgemm_i8_quantize takes: 2^24 - 1 rows, four times as many of
 * K up to 1024, 16 times as many of K up to 256.
 */
int sgemm_i8_quantize(int dtype, int M, int K, const void *X, int ldx,
                      void *values, int ldv, float *scales, void *stream);
int sgemm_i8_dequantize(int dtype, int M, int K, const void *values, int ldv, const float *scales,
                        void *X, int ldx, void *stream);

/*
 * sgemm_grouped_sort: T tokens, each with `picks` experts, sorted by expert into
 * n = T * picks rows for the grouped products.  experts[t * lde + j], of
 * expert_bytes (4 or 8) bytes, is the expert of token t's pick j; any value
 * outside 0 .. groups - 1 stands for no group (a padded token, another rank's
 * expert).  Written are
 *   offsets   [groups + 1]  rows offsets[g] .. offsets[g+1] - 1 are group g's, by
 *                           token, then by pick
 *   position  [T][picks]    the row of (t, j), or -1 for no group
 *   source    [n]           t * picks + j of each row, -1 behind offsets[groups]
 *   rows      [n,H]         row position[t][j] is X[t]; zeros behind
 *                           offsets[groups].  NULL: not wanted
 * X [T,H] of BF16, FP16, FP32 or SGEMM_DTYPE_I8; with the last x_scales [T] are
 * brought to row_scales [n] in the same way (not where rows is NULL, but if H is
 * 0: rows of no columns have no address).  groups up to 4096, n below 2^31 - 1,
 * H up to 2^28.  The gradient with respect to X is
 * sgemm_grouped_combine() without weights.
 *
 * sgemm_grouped_combine: the way back,
 *   out[t] = sum_j weights[t * ldw + j] * Y[position[t][j]],
 * summed in FP32 in the order of j, picks of no group left out; weights of
 * dtype_w (BF16, FP16 or FP32), NULL: 1.  Y [n,H], out [T,H]: of one type, or
 * one of them FP32.
 *
 * sgemm_grouped_combine_grad: for D, the gradient with respect to out,
 *   dY[position[t][j]] = weights[t * ldw + j] * D[t],
 *   dweights[t][j] = sum_h D[t][h] * Y[position[t][j]][h],
 * dY [n,H] of Y's type, zeros behind offsets[groups], dweights [T][picks] of
 * dtype_w, 0 for picks of no group; either may be NULL if it is not wanted (Y
 * is read for dweights only).  D and Y: of one type, or one of them FP32.
 */
int sgemm_grouped_sort(int dtype, int T, int picks, int groups, int H,
                       const void *X, int ldx, const float *x_scales,
                       const void *experts, int lde, int expert_bytes,
                       int *offsets, int *position, int *source,
                       void *rows, int ldr, float *row_scales,
                       void *workspace, long long workspace_bytes, void *stream);
long long sgemm_grouped_sort_workspace(int T, int picks, int groups);
int sgemm_grouped_combine(int dtype, int dtype_out, int T, int picks, int H,
                          const void *Y, int ldy, const int *position,
                          const void *weights, int ldw, int dtype_w,
                          void *out, int ldo, void *stream);
int sgemm_grouped_combine_grad(int dtype, int dtype_d, int T, int picks, int groups, int H,
                               const void *D, int ldd, const void *Y, int ldy,
                               const int *offsets, const int *position,
                               const void *weights, int ldw, int dtype_w,
                               void *dY, int lddy, void *dweights, void *stream);

/* The variant sgemm_lowp() would run for these arguments (no launch; the
 * pointers are only inspected for alignment), or SGEMM_STATUS_INVALID_DIM.
 * 0 (the plain kernel) also where sgemm_lowp() copies the operands and runs
 * a fast kernel on the copies. */
int sgemm_lowp_select_variant(int M, int N, int K,
                              const void *A, int lda,
                              const void *B, int ldb);

/* Split-K factor (1 = no split) that sgemm_lowp_ex() with this variant would
 * use for an M x N x K problem outside graph capture; no HIP call.  (A strided
 * batch of untransposed problems counts its problems' tiles together; the
 * environment variable SGEMM_SPLITK = S caps the factor at S, for sweeps.)
 * Returns the factor, SGEMM_STATUS_INVALID_VARIANT or
 * SGEMM_STATUS_INVALID_DIM. */
int sgemm_lowp_split_factor(int variant, int M, int N, int K);

/* Static name of a sgemm_lowp_ex() variant, or NULL for an unknown id. */
const char *sgemm_lowp_variant_name(int variant);

/*
 * sgemm_split_factor: the number of workgroups per output tile along K
 * (1 = no split) that sgemm_ex() with this variant would use for an
 * M x N x K problem whose operands the variant's split-K kernel takes (see
 * "Workspace" above; environment variable SGEMM_SPLITK = S forces S for
 * sweeps).  Only grids of fewer than 512 tiles split; the factor (at most
 * 16, at least two K tiles per split) is the one of least modelled kernel
 * time: the busiest compute unit's share of K tiles plus a fixed cost per
 * pair of resident blocks, bounded below by the grid's operand traffic,
 * plus a fixed cost of splitting and one per split (the partials read
 * back); taken when that is at most 95% of the unsplit time.  The model's
 * constants are fitted to kernel-trace durations of 46 small grids at up
 * to 12 factors each.  Always 1 for variants
 * without split-K.  No HIP call.  Returns the factor,
 * SGEMM_STATUS_INVALID_VARIANT or SGEMM_STATUS_INVALID_DIM (negative sizes).
 */
int sgemm_split_factor(int variant, int M, int N, int K);

/*
 * sgemm_tail_split: the split of the last wave that sgemm_ex() with this
 * variant would make for an M x N x K problem with packed leading dimensions
 * outside graph capture (no HIP call).  A split-capable variant whose grid
 * is whole waves of tiles (two workgroups per compute unit) plus a partly
 * filled last wave, and that does not split K already, runs as two launches
 * on the stream when the same cost model as sgemm_split_factor (plus a fixed
 * cost for the second launch) says that saves at least 5%: the whole waves,
 * then the last wave's tiles with K split S ways.  Returns S (1: a single
 * launch) and, if tail_tiles is not
 * NULL, stores the number of tiles in the second launch (0 when S is 1);
 * SGEMM_STATUS_INVALID_VARIANT or SGEMM_STATUS_INVALID_DIM on bad arguments.
 */
int sgemm_tail_split(int variant, int M, int N, int K, int *tail_tiles);

/*
 * sgemm_workspace_bytes: device memory (bytes) the library holds on the
 * current device for split-K workspaces and copy buffers; at most
 * SGEMM_MAX_STREAM_WORKSPACES * SGEMM_WORKSPACE_BYTES + SGEMM_MAX_COPY_BUFFERS
 * * SGEMM_MAX_COPY_BUFFER_BYTES.  SGEMM_STATUS_HIP_ERROR if the current
 * device cannot be read.
 */
long long sgemm_workspace_bytes(void);

/*
 * sgemm_release_workspaces: free the workspaces and copy buffers the library
 * holds on the current device, each after the kernels queued with it have
 * finished (this call waits for them: on an event where one marks the last
 * use, else once for the whole device, hipDeviceSynchronize).  Buffers held by calls in progress on
 * other host threads at that moment are left alone.  Later calls allocate
 * again as needed.  Returns SGEMM_STATUS_OK or SGEMM_STATUS_HIP_ERROR (a
 * buffer whose wait or free failed is kept and never reused).
 */
int sgemm_release_workspaces(void);

/* Static text for a status code. */
const char *sgemm_strerror(int status);

/* Text of the last HIP error seen by this thread ("" if none). */
const char *sgemm_last_hip_error(void);

/* Library version (monotonic integer). */
int sgemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MI355X_H */

// Products grouped by rows, 16-bit inputs with FP32 accumulation: the rows
// of A are in groups (offsets[g] .. offsets[g+1], read on the device), each
// with a matrix B[g] of its own.
//
//   group_rows_kernel,
//   group_mixed_kernel  C[rows of g] = alpha * A[rows of g] * op(B[g]) + beta * C
//   group_k_kernel      C[g] = alpha * A[rows of g]^T * D[rows of g] + beta * C[g]
//
// They run the K loop of sgemm_lowp.hpp on one block tile.  The host does
// not know the groups' sizes, so the first kernels' grids cover the most
// tiles that any split of the rows can have, floor((M + g*(BM-1)) / BM) tile
// rows for g = min(groups, M) groups, and a workgroup finds its tile from
// the offsets (one wave-wide scan of the groups' tile counts); workgroups
// past the last tile end at once.
#include <algorithm>

#include "sgemm_tile16.hpp"

namespace sgemm_mi355x {

struct GroupArgs {
    const char *A, *B;
    char *C;
    long lda, ldb, ldc, strideB, strideC;   // elements
    const int *offsets;
    int groups, M, N, K;                    // M: rows of A
    float alpha, beta;
};

// Rows of group g, clamped to 0 .. M whatever the offsets hold.
__device__ __forceinline__ void group_rows(const int *offsets, int g, int M, int &lo, int &rows) {
    lo = min(max(offsets[g], 0), M);
    rows = min(max(offsets[g + 1], lo), M) - lo;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The groups' tiles of BM rows one after another: how many there are, at most
// `most`, and the group and the tile of number `id`.  Wave-uniform.  (Groups that
// overlap, in offsets that decrease, can have more tiles than the grid covers and
// than 32 bits count: products with the number of tile columns are formed in 64.
// The tile rows of 64 groups fit 32 bits: 64 * 2^31 / 256, and M is at most 65535
// times 32 or 128 where BM is less.)
template <int BM>
struct TileList {
    const GroupArgs &p;
    int tiles_n, first, total;                  // first: tile rows of group `lane`
    __device__ __forceinline__ int tile_rows(int g) const {
        int l = 0, r = 0;
        if (g < p.groups) group_rows(p.offsets, g, p.M, l, r);
        return (r + BM - 1) / BM;
    }
    __device__ __forceinline__ TileList(const GroupArgs &args, int bn, int most) : p(args), tiles_n((args.N + bn - 1) / bn) {
        const int lane = threadIdx.x & 63;
        first = tile_rows(lane);
        long sum = __builtin_amdgcn_readfirstlane(wave_sum(first));
        for (int base = 64; base < p.groups; base += 64) sum += __builtin_amdgcn_readfirstlane(wave_sum(tile_rows(base + lane)));
        total = (int)min(sum * tiles_n, (long)most);
    }
    // (id < total)
    __device__ __forceinline__ void find(int id, int &g, int &lo, int &rows, int &tm, int &tn) const {
        const int lane = threadIdx.x & 63;
        for (int base = 0; base < p.groups; base += 64) {
            const int mine = base ? tile_rows(base + lane) : first;
            int upto = mine;                                    // tile rows up to this lane's group
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int below = __shfl_up(upto, d);
                if (lane >= d) upto += below;
            }
            const unsigned long past = __ballot(id < (long)upto * tiles_n);
            if (past) {
                const int at = __builtin_ctzl(past);
                const int count = __builtin_amdgcn_readlane(mine, at);
                id -= (__builtin_amdgcn_readlane(upto, at) - count) * tiles_n;
                group_rows(p.offsets, base + at, p.M, lo, rows);
                g = __builtin_amdgcn_readfirstlane(base + at);
                lo = __builtin_amdgcn_readfirstlane(lo);
                rows = __builtin_amdgcn_readfirstlane(rows);
                raster(id, count, tiles_n, tm, tn);
                return;
            }
            id -= __builtin_amdgcn_readlane(upto, 63) * tiles_n;
        }
    }
};

template <class T, bool F16, bool TB, bool OUT16>
__device__ __forceinline__ void group_tile(const GroupArgs &p, char *lds, int g, int lo, int rows, int m0, int n0) {
    const Operands16 q = {p.A + 2L * lo * p.lda, p.B + 2L * g * p.strideB, p.lda, p.ldb, rows, p.N, p.K};
    f32x4 acc[T::MI][T::NB];
    accumulate16<T, F16, false, TB>(q, m0, n0, lds, acc);
    store_tile<T, F16, OUT16>(acc, m0, n0, rows, p.N, p.C + (OUT16 ? 2L : 4L) * lo * p.ldc, p.ldc, p.alpha, p.beta);
}

// One tile shape throughout.
template <class T, bool F16, bool TB, bool OUT16>
__global__ void __launch_bounds__(T::NT) group_rows_kernel(GroupArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[T::LDS];
    const TileList<T::BM> list(p, T::BN, gridDim.x);
    if ((int)blockIdx.x >= list.total) return;
    int g = 0, lo = 0, rows = 0, tm = 0, tn = 0;
    list.find(xcd_run(blockIdx.x, list.total), g, lo, rows, tm, tn);
    if (tm * T::BM < rows) group_tile<T, F16, TB, OUT16>(p, lds, g, lo, rows, tm * T::BM, tn * T::BN);
}

// Tiles of 256 x 256 with a finer last round.
template <bool F16, bool TB, bool OUT16>
struct GroupBody {
    const TileList<256> list;
    template <class T>
    __device__ __forceinline__ void tile(char *lds, int id, int sub) const {
        int g = 0, lo = 0, rows = 0, tm = 0, tn = 0, m0, n0;
        list.find(id, g, lo, rows, tm, tn);
        part_corner<T>(tm, tn, sub, m0, n0);
        if (m0 < rows && n0 < list.p.N) group_tile<T, F16, TB, OUT16>(list.p, lds, g, lo, rows, m0, n0);
    }
};

template <bool F16, bool TB, bool OUT16>
__global__ void __launch_bounds__(512) group_mixed_kernel(GroupArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[Mixed<TB>::LDS];
    const GroupBody<F16, TB, OUT16> body{TileList<256>(p, 256, gridDim.x - mixed_grid(0))};
    Mixed<TB>::run(body, lds, body.list.total);
}

// The group of `turn` when up to 64 groups go by their rows, most first.
__device__ __forceinline__ int longest_first(const GroupArgs &p, int turn) {
    const int lane = threadIdx.x & 63;
    int lo, mine = -1, rank = 0;
    if (lane < p.groups) group_rows(p.offsets, lane, p.M, lo, mine);
    for (int j = 0; j < p.groups; ++j) {
        const int other = __builtin_amdgcn_readlane(mine, j);
        rank += other > mine || (other == mine && j < lane);
    }
    return __builtin_ctzl(__ballot(lane < p.groups && rank == turn));
}

// A [M][K] and B [M][N] by rows; C[g] is K x N, the sum runs over the
// group's rows.  A group's tiles go round the XCDs in runs of their own, so
// that uneven groups still load the XCDs evenly, and the longest groups go
// first, so that the last tiles to run are short ones.  Block y of gridDim.y
// takes its share of the group's rows, into C's of its own.
template <class T, bool F16, bool OUT16>
__global__ void __launch_bounds__(T::NT) group_k_kernel(GroupArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[T::LDS];
    const int tiles_m = (p.K + T::BM - 1) / T::BM, tiles_n = (p.N + T::BN - 1) / T::BN;
    const int tiles = tiles_m * tiles_n, per = (tiles + 7) >> 3;
    const int turn = blockIdx.x / (8 * per), id = (blockIdx.x & 7) * per + (blockIdx.x - turn * 8 * per >> 3);
    if (id >= tiles) return;
    int lo, rows, tm, tn;
    const int g = p.groups <= 64 ? longest_first(p, turn) : turn;
    group_rows(p.offsets, g, p.M, lo, rows);
    lo = __builtin_amdgcn_readfirstlane(lo);
    rows = __builtin_amdgcn_readfirstlane(rows);
    raster(id, tiles_m, tiles_n, tm, tn);
    const int shares = gridDim.y, part = (rows + 64 * shares - 1) / (64 * shares) * 64;        // whole K tiles
    lo += min(part * (int)blockIdx.y, rows);
    rows = min(part, max(rows - part * (int)blockIdx.y, 0));
    const Operands16 q = {p.A + 2L * lo * p.lda, p.B + 2L * lo * p.ldb, p.lda, p.ldb, p.K, p.N, rows};
    f32x4 acc[T::MI][T::NB];
    accumulate16<T, F16, true, false>(q, tm * T::BM, tn * T::BN, lds, acc);
    const long at = g + (long)blockIdx.y * p.groups;
    store_tile<T, F16, OUT16>(acc, tm * T::BM, tn * T::BN, p.K, p.N, p.C + (OUT16 ? 2L : 4L) * at * p.strideC, p.ldc,
                              p.alpha, p.beta);
}

// C = alpha * the sum of the shares' products + beta * C, the shares in order;
// a thread per four columns.
template <bool F16, bool OUT16>
__global__ void __launch_bounds__(256) group_join_kernel(GroupArgs p, const float *parts, long ld, int shares) {
    const long quads = (p.N + 3) / 4, t = blockIdx.x * 256L + threadIdx.x;
    if (t >= quads * p.K * p.groups) return;
    const long row = t / quads, g = row / p.K;              // row: of all groups' matrices
    const int col = 4 * (int)(t - row * quads);
    const f32x4 v = sum_shares(parts + row * ld + col, (long)p.groups * p.K * ld, shares);
    store4<F16, OUT16>(p.C + (OUT16 ? 2L : 4L) * (g * p.strideC + (row - g * p.K) * p.ldc), col, p.N, p.beta, v * p.alpha);
}

// One 16-byte chunk of dst per thread and step, a row per workgroup and step,
// from rows of any alignment (a 16-byte load needs none on this chip; the copy is
// bound by memory).
__global__ void __launch_bounds__(256) pad_rows_kernel(const unsigned short *src, long ld, long stride, int rows,
                                                       int cols, unsigned short *dst, int chunks) {
    typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
    src += blockIdx.y * stride;
    dst += (long)blockIdx.y * rows * chunks * 8;
    for (long r = blockIdx.x; r < rows; r += gridDim.x) {
        const unsigned short *from = src + r * ld;
        for (int q = threadIdx.x; q < chunks; q += 256) {
            const int c = 8 * q;
            u16x8 v;
            if (c + 8 <= cols) {
                __builtin_memcpy(&v, from + c, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? from[c + e] : (unsigned short)0;
            }
            reinterpret_cast<u16x8 *>(dst)[r * chunks + q] = v;
        }
    }
}

hipError_t pad_rows(const void *src, long ld, long stride, int copies, int rows, int cols, void *dst, hipStream_t s) {
    return launch_k(pad_rows_kernel, dim3((unsigned)std::min(rows, 1 << 22), (unsigned)copies), dim3(256), s,
                    static_cast<const unsigned short *>(src), ld, stride, rows, cols, static_cast<unsigned short *>(dst),
                    (cols + 7) / 8);
}

namespace {

constexpr int kMaxGroups = 65535;   // launch grid extent of the padded copies

// KERNEL<before..., F16, after..., OUT16>
#define GROUP_FORMS(KERNEL, NT, BEFORE, AFTER)                                                  \
    (f16 ? (out16 ? launch_k(KERNEL<BEFORE true, AFTER true>, grid, dim3(NT), s, p)             \
                  : launch_k(KERNEL<BEFORE true, AFTER false>, grid, dim3(NT), s, p))           \
         : (out16 ? launch_k(KERNEL<BEFORE false, AFTER true>, grid, dim3(NT), s, p)            \
                  : launch_k(KERNEL<BEFORE false, AFTER false>, grid, dim3(NT), s, p)))
#define COMMA ,

// The most tiles of bm x bn that any split of the rows into groups can have.
long most_tiles(const GroupArgs &p, int bm, int bn) {
    const long groups = std::min(p.groups, p.M);
    return (p.M + groups * (bm - 1)) / bm * ((p.N + bn - 1) / bn);
}

template <class T, bool TB>
hipError_t launch_rows(const GroupArgs &p, bool f16, bool out16, hipStream_t s) {
    const dim3 grid((unsigned)most_tiles(p, T::BM, T::BN));
    return GROUP_FORMS(group_rows_kernel, T::NT, T COMMA, TB COMMA);
}

template <bool TB>
hipError_t launch_mixed(const GroupArgs &p, bool f16, bool out16, hipStream_t s) {
    const dim3 grid((unsigned)mixed_grid(most_tiles(p, 256, 256)));
    return GROUP_FORMS(group_mixed_kernel, 512, , TB COMMA);
}

template <class T>
hipError_t launch_wgrad(const GroupArgs &p, int shares, bool f16, bool out16, hipStream_t s) {
    const long tiles = (long)((p.K + T::BM - 1) / T::BM) * ((p.N + T::BN - 1) / T::BN);
    const dim3 grid((unsigned)(ceil_to(tiles, 8) * p.groups), (unsigned)shares);
    return GROUP_FORMS(group_k_kernel, T::NT, T COMMA, );
}

// Whether launch_rows() can cover M rows.
bool rows_fit(int groups, int M, int N) {
    GroupArgs p = {};
    p.groups = groups;
    p.M = M;
    p.N = N;
    const int rows = groups > 0 && M > 0 ? M / std::min(groups, M) : 0;
    return rows <= 32    ? launch_fits(most_tiles(p, 32, 128), Tile32::NT)
           : rows <= 128 ? launch_fits(most_tiles(p, 128, 128), Tile128::NT)
                         : launch_fits(mixed_grid(most_tiles(p, 256, 256)), 512);
}

// By the rows of an average group: tiles of 32 rows are bound by the weights'
// bytes, tiles of 128 leave less of a small group empty, tiles of 256 load
// least.
hipError_t launch_rows(const GroupArgs &p, bool tb, bool f16, bool out16, hipStream_t s) {
    const int rows = p.M / std::min(p.groups, p.M);
    if (rows <= 32) return tb ? launch_rows<Tile32, true>(p, f16, out16, s) : launch_rows<Tile32, false>(p, f16, out16, s);
    if (rows <= 128) return tb ? launch_rows<Tile128, true>(p, f16, out16, s) : launch_rows<Tile128, false>(p, f16, out16, s);
    return tb ? launch_mixed<true>(p, f16, out16, s) : launch_mixed<false>(p, f16, out16, s);
}

// Shares of the rows of each group: small matrices over many rows would leave
// most of the chip idle, so as many as fill it, of 256 rows of an average group
// at least (6984 rows in 2 groups, 192 x 656 each: 39.5 -> 19 us).
int wgrad_shares(int groups, int M, int N, int K) {
    const long tiles = (K + 127L) / 128 * ((N + 127L) / 128) * std::max(groups, 1);
    return (int)std::max(1L, std::min(512 / std::max(tiles, 1L), M / std::max(groups, 1) / 256L));
}

long join_bytes(int groups, int M, int N, int K) {          // the shares' FP32 products
    const int shares = wgrad_shares(groups, M, N, K);
    return shares > 1 ? 4L * shares * groups * K * ceil_to(N, 4) : 0;
}

// Fewer than a round of the large tiles: the next smaller that fill it.
hipError_t launch_wgrad(const GroupArgs &p, float *parts, bool f16, bool out16, hipStream_t s) {
    const int shares = wgrad_shares(p.groups, p.M, p.N, p.K);
    if (shares > 1) {
        GroupArgs q = p;
        q.C = reinterpret_cast<char *>(parts);
        q.ldc = ceil_to(p.N, 4);
        q.strideC = p.K * q.ldc;
        q.alpha = 1.f;
        q.beta = 0.f;
        const hipError_t e = launch_wgrad<Tile128>(q, shares, f16, false, s);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)(((p.N + 3L) / 4 * p.K * p.groups + 255) / 256)), block(256);
        if (f16) return out16 ? launch_k(group_join_kernel<true, true>, grid, block, s, p, parts, q.ldc, shares)
                              : launch_k(group_join_kernel<true, false>, grid, block, s, p, parts, q.ldc, shares);
        return out16 ? launch_k(group_join_kernel<false, true>, grid, block, s, p, parts, q.ldc, shares)
                     : launch_k(group_join_kernel<false, false>, grid, block, s, p, parts, q.ldc, shares);
    }
    const long n256 = (p.N + 255) / 256, m128 = (p.K + 127) / 128;
    if ((p.K + 255) / 256 * n256 * p.groups >= 256) return launch_wgrad<Tile256>(p, 1, f16, out16, s);
    if (m128 * n256 * p.groups >= 256) return launch_wgrad<TileWide>(p, 1, f16, out16, s);
    return launch_wgrad<Tile128>(p, 1, f16, out16, s);
}

bool in_dtype(int d) { return d == SGEMM_DTYPE_BF16 || d == SGEMM_DTYPE_F16; }

// Bytes of the zero-padded copies of the operands whose rows are not whole
// aligned 16-byte chunks; 0 for an operand that is taken as it is.  (A chunk
// that straddles K holds zeros in the copy, and the K loop reads rows of an
// untransposed B past K as zeros.)
struct Copies {
    long a, b;
};

Copies rows_copies(bool tb, int groups, int M, int N, int K, const void *A, int lda, const void *B, int ldb,
                   long long stride_b) {
    const bool a = !chunk_rows(A, lda, K), b = !chunk_rows(B, ldb, tb ? K : N) || (groups > 1 && stride_b % 8 != 0);
    return {a ? ceil_to(2L * M * ceil_to(K, 8), 256) : 0,
            b ? 2L * groups * (tb ? N * ceil_to(K, 8) : K * ceil_to(N, 8)) : 0};
}

Copies k_copies(int M, int N, int K, const void *A, int lda, const void *D, int ldd) {
    return {chunk_rows(A, lda, K) ? 0 : ceil_to(2L * M * ceil_to(K, 8), 256),
            chunk_rows(D, ldd, N) ? 0 : ceil_to(2L * M * ceil_to(N, 8), 256)};
}

bool scratch_ok(long need, const void *workspace, long long bytes) {
    return need == 0 || (workspace != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(workspace) & 15) == 0);
}

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

long long sgemm_lowp_grouped_workspace(int op_b, int groups, int M, int N, int K, const void *A, int lda, const void *B,
                                       int ldb, long long stride_b) {
    if (op_b != SGEMM_OP_N && op_b != SGEMM_OP_T) return SGEMM_STATUS_INVALID_OP;
    if (groups < 0 || M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    if (groups == 0 || M == 0 || N == 0 || K == 0) return 0;
    const Copies c = rows_copies(op_b == SGEMM_OP_T, groups, M, N, K, A, lda, B, ldb, stride_b);
    return c.a + c.b;
}

int sgemm_lowp_grouped(int dtype, int op_b, int groups, int M, int N, int K, float alpha, const void *A, int lda,
                       const void *B, int ldb, long long stride_b, const int *offsets, float beta, void *C, int ldc,
                       int dtype_c, void *workspace, long long workspace_bytes, void *stream) {
    if (!in_dtype(dtype) || (dtype_c != dtype && dtype_c != SGEMM_DTYPE_F32)) return SGEMM_STATUS_INVALID_DTYPE;
    if (op_b != SGEMM_OP_N && op_b != SGEMM_OP_T) return SGEMM_STATUS_INVALID_OP;
    const bool tb = op_b == SGEMM_OP_T, f16 = dtype == SGEMM_DTYPE_F16, out16 = dtype_c != SGEMM_DTYPE_F32;
    if (groups < 0 || groups > kMaxGroups || M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    if (lda < std::max(K, 1) || ldb < std::max(tb ? K : N, 1) || ldc < std::max(N, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (stride_b < 0 || K > kMaxLd16 || N > kMaxLd16) return SGEMM_STATUS_INVALID_DIM;
    if (!rows_fit(groups, M, N)) return SGEMM_STATUS_INVALID_DIM;
    if (groups == 0 || M == 0 || N == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || offsets == nullptr || (K > 0 && (A == nullptr || B == nullptr))) return SGEMM_STATUS_NULL_POINTER;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    GroupArgs p = {static_cast<const char *>(A), static_cast<const char *>(B), static_cast<char *>(C), lda, ldb, ldc,
                   stride_b, 0, offsets, groups, M, N, K, alpha, beta};
    if (K > 0) {
        const Copies c = rows_copies(tb, groups, M, N, K, A, lda, B, ldb, stride_b);
        if (!scratch_ok(c.a + c.b, workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
        char *w = static_cast<char *>(workspace);
        hipError_t e = hipSuccess;
        if (c.a) {
            e = pad_rows(A, lda, 0, 1, M, K, w, s);
            p.A = w;
            p.lda = ceil_to(K, 8);
        }
        if (e == hipSuccess && c.b) {
            const int rows = tb ? N : K, cols = tb ? K : N;
            e = pad_rows(B, ldb, stride_b, groups, rows, cols, w + c.a, s);
            p.B = w + c.a;
            p.ldb = ceil_to(cols, 8);
            p.strideB = rows * p.ldb;
        }
        if (e != hipSuccess) return hip_status(e, "kernel launch");
    }
    const hipError_t e = launch_rows(p, tb, f16, out16, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

long long sgemm_lowp_grouped_wgrad_workspace(int groups, int M, int N, int K, const void *A, int lda, const void *D,
                                             int ldd) {
    if (groups < 0 || M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    if (groups == 0 || M == 0 || N == 0 || K == 0) return 0;
    const Copies c = k_copies(M, N, K, A, lda, D, ldd);
    return c.a + c.b + join_bytes(groups, M, N, K);
}

int sgemm_lowp_grouped_wgrad(int dtype, int groups, int M, int N, int K, float alpha, const void *A, int lda,
                             const void *D, int ldd, const int *offsets, float beta, void *C, int ldc,
                             long long stride_c, int dtype_c, void *workspace, long long workspace_bytes,
                             void *stream) {
    if (!in_dtype(dtype) || (dtype_c != dtype && dtype_c != SGEMM_DTYPE_F32)) return SGEMM_STATUS_INVALID_DTYPE;
    const bool f16 = dtype == SGEMM_DTYPE_F16, out16 = dtype_c != SGEMM_DTYPE_F32;
    if (groups < 0 || groups > kMaxGroups || M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    if (lda < std::max(K, 1) || ldd < std::max(N, 1) || ldc < std::max(N, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (K > kMaxLd16 || N > kMaxLd16) return SGEMM_STATUS_INVALID_DIM;
    if (groups > 1 && K > 0 && N > 0 && stride_c < (K - 1LL) * ldc + N) return SGEMM_STATUS_INVALID_DIM;
    if (!launch_fits(ceil_to((K + 127L) / 128 * ((N + 127L) / 128), 8) * groups, TileWide::NT)) return SGEMM_STATUS_INVALID_DIM;
    if (groups == 0 || N == 0 || K == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || offsets == nullptr || (M > 0 && (A == nullptr || D == nullptr))) return SGEMM_STATUS_NULL_POINTER;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    GroupArgs p = {static_cast<const char *>(A), static_cast<const char *>(D), static_cast<char *>(C), lda, ldd, ldc,
                   0, stride_c, offsets, groups, M, N, K, alpha, beta};
    char *w = static_cast<char *>(workspace);
    const Copies c = M > 0 ? k_copies(M, N, K, A, lda, D, ldd) : Copies{0, 0};
    if (!scratch_ok(c.a + c.b + join_bytes(groups, M, N, K), workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    if (M > 0) {
        hipError_t e = hipSuccess;
        if (c.a) {
            e = pad_rows(A, lda, 0, 1, M, K, w, s);
            p.A = w;
            p.lda = ceil_to(K, 8);
        }
        if (e == hipSuccess && c.b) {
            e = pad_rows(D, ldd, 0, 1, M, N, w + c.a, s);
            p.B = w + c.a;
            p.ldb = ceil_to(N, 8);
        }
        if (e != hipSuccess) return hip_status(e, "kernel launch");
    }
    const hipError_t e = launch_wgrad(p, reinterpret_cast<float *>(w + c.a + c.b), f16, out16, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

}  // extern "C"

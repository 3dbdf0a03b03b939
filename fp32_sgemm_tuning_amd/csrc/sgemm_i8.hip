// Products of 8-bit integers with a scale for each row of X (a token) and each
// row of W (an output channel),
//   C[m][n] = alpha * sx[m] * sw[n] * sum_k x[m][k] * w[n][k] + beta * C[m][n],
// of one weight or of one weight per group of rows, and the kernels that bring
// a matrix into that form and back.
//
// The sums are exact: 32-bit integers hold K * 128 * 128 for K < 2^17.  So K may
// be split in any way and the result is rounded by the scales alone:
// ((float)sum * (alpha * sx)) * sw, in FP32, then to C's type.
//
//   i8_rows_kernel   few rows of X: bound by W's bytes
//   i8_tile_kernel,
//   i8_mixed_kernel  tiles through LDS, on the K loop of sgemm_lowp.hpp
//   i8_join_kernel   adds the shares of a split K
//   i8_quantize_kernel, i8_dequantize_kernel
#include <algorithm>
#include <type_traits>

#include "sgemm_rows.hpp"

namespace sgemm_mi355x {

namespace {

struct I8Args {
    const char *X, *W;                      // 8-bit integers, rows of whole aligned 16-byte chunks
    const float *sx, *sw;
    char *C;
    long ldx, ldw, ldc, strideW, strideS;   // elements; strides from group to group
    const int *offsets;                     // NULL: one group of all rows
    int groups, M, N, K;
    float alpha, beta;
    int dtype_c;
    int *parts;                             // the shares' sums [shares][M][ceil_to(N, 4)]
    __device__ __forceinline__ void rows_of(int g, int &lo, int &rows) const {
        if (offsets) group_rows(offsets, g, M, lo, rows);
        else lo = 0, rows = M;
    }
};

// The operands of one tile's product as lowp_accumulate takes them: pairs of
// integers, K up to whole chunks, `cut` bytes of the last (0: all).
struct Operands8 {
    const char *A, *B;
    long lda, ldb;
    int M, N, K, cut;
};

template <class T, bool SPLIT>
__device__ __forceinline__ void accumulate8(const Operands8 &q, int m0, int n0, char *lds, int S, int y, i32x4 (&acc)[T::MI][T::NB]) {
    lowp_accumulate<T::BM, T::BN, T::BK, T::WAVES_M, T::WAVES_N, T::NS, T::PP, true, kMulI8, SPLIT, false, true>(
        q, m0, n0, lds, S, y, acc);
}

__device__ __forceinline__ f32x4 to_float(i32x4 v) { return __builtin_convertvector(v, f32x4); }

// Four scales from `at` on, those from N on taken as 0.
__device__ __forceinline__ f32x4 scales4(const float *sw, int at, int N) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (at + 3 < N) {
        __builtin_memcpy(&s, sw + at, 16);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (at + r < N) s[r] = sw[at + r];
    }
    return s;
}

// f(fp16, 16-bit) for the result's type.
template <class F>
__device__ __forceinline__ void by_result(int dtype, F &&f) {
    if (dtype == SGEMM_DTYPE_F32) f(std::false_type{}, std::false_type{});
    else if (dtype == SGEMM_DTYPE_BF16) f(std::false_type{}, std::true_type{});
    else f(std::true_type{}, std::true_type{});
}

// The tile at (m0, n0) of a product of `rows` rows from row lo on, scaled.
template <class T>
__device__ __forceinline__ void store_scaled(const I8Args &p, const i32x4 (&acc)[T::MI][T::NB], int g, int lo, int rows, int m0, int n0) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float *sw = p.sw + g * p.strideS;
    const int col0 = n0 + (wave % T::WAVES_N) * T::WN + 4 * (lane >> 4);
    f32x4 s[T::NB];
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) s[nb] = scales4(sw, col0 + 16 * nb, p.N);
    by_result(p.dtype_c, [&](auto f16, auto out16) {
        constexpr int E = decltype(out16)::value ? 2 : 4;
#pragma unroll
        for (int mi = 0; mi < T::MI; ++mi) {
            const int row = m0 + (wave / T::WAVES_N) * T::WM + mi * 16 + (lane & 15);
            if (row >= rows) continue;
            const float sx = p.alpha * p.sx[lo + row];
            char *to = p.C + (long)(lo + row) * p.ldc * E;
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb)
                store4<decltype(f16)::value, decltype(out16)::value>(to, col0 + 16 * nb, p.N, p.beta, to_float(acc[mi][nb]) * sx * s[nb]);
        }
    });
}

template <class T>
__device__ __forceinline__ void i8_tile(const I8Args &p, char *lds, int g, int lo, int rows, int m0, int n0) {
    const Operands8 q = {p.X + lo * p.ldx, p.W + g * p.strideW, p.ldx >> 1, p.ldw >> 1, rows, p.N, (p.K + 15) / 16 * 8, p.K & 15};
    i32x4 acc[T::MI][T::NB];
    accumulate8<T, false>(q, m0, n0, lds, 1, 0, acc);
    store_scaled<T>(p, acc, g, lo, rows, m0, n0);
}

// One tile shape throughout.
template <class T>
__global__ void __launch_bounds__(T::NT) i8_tile_kernel(I8Args p) {
    __shared__ __attribute__((aligned(16))) char lds[T::LDS];
    const TileList<T::BM, I8Args> list(p, T::BN, gridDim.x);
    if ((int)blockIdx.x >= list.total) return;
    int g = 0, lo = 0, rows = 0, tm = 0, tn = 0;
    list.find(xcd_run(blockIdx.x, list.total), g, lo, rows, tm, tn);
    if (tm * T::BM < rows) i8_tile<T>(p, lds, g, lo, rows, tm * T::BM, tn * T::BN);
}

// Tiles of 256 x 256 with a finer last round.
struct I8Body {
    const TileList<256, I8Args> list;
    template <class T>
    __device__ __forceinline__ void tile(char *lds, int id, int sub) const {
        int g = 0, lo = 0, rows = 0, tm = 0, tn = 0, m0, n0;
        list.find(id, g, lo, rows, tm, tn);
        part_corner<T>(tm, tn, sub, m0, n0);
        if (m0 < rows && n0 < list.p.N) i8_tile<T>(list.p, lds, g, lo, rows, m0, n0);
    }
};

__global__ void __launch_bounds__(512) i8_mixed_kernel(I8Args p) {
    __shared__ __attribute__((aligned(16))) char lds[Mixed<true>::LDS];
    const I8Body body{TileList<256, I8Args>(p, 256, gridDim.x - mixed_grid(0))};
    Mixed<true>::run(body, lds, body.list.total);
}

// One weight, share blockIdx.y of gridDim.y of K: its sums, for i8_join_kernel.
template <class T>
__global__ void __launch_bounds__(T::NT) i8_share_kernel(I8Args p) {
    __shared__ __attribute__((aligned(16))) char lds[T::LDS];
    const int tiles_m = (p.M + T::BM - 1) / T::BM, tiles_n = (p.N + T::BN - 1) / T::BN;
    int tm, tn;
    raster(xcd_run(blockIdx.x, gridDim.x), tiles_m, tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    const Operands8 q = {p.X, p.W, p.ldx >> 1, p.ldw >> 1, p.M, p.N, (p.K + 15) / 16 * 8, p.K & 15};
    i32x4 acc[T::MI][T::NB];
    accumulate8<T, true>(q, m0, n0, lds, gridDim.y, blockIdx.y, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long ld = (p.N + 3L) / 4 * 4;
    int *to = p.parts + (long)blockIdx.y * p.M * ld;
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
        const int row = m0 + (wave / T::WAVES_N) * T::WM + mi * 16 + (lane & 15);
        if (row >= p.M) continue;
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) {
            const int col = n0 + (wave % T::WAVES_N) * T::WN + nb * 16 + 4 * (lane >> 4);
            if (col < ld) *reinterpret_cast<i32x4 *>(to + row * ld + col) = acc[mi][nb];
        }
    }
}

// C from the shares' sums; a thread per four columns.
__global__ void __launch_bounds__(256) i8_join_kernel(I8Args p, int shares) {
    const long quads = (p.N + 3L) / 4, t = blockIdx.x * 256L + threadIdx.x;
    if (t >= quads * p.M) return;
    const long row = t / quads, step = p.M * quads * 4;
    const int col = 4 * (int)(t - row * quads);
    i32x4 v = {0, 0, 0, 0};
    for (int y = 0; y < shares; ++y) v += *reinterpret_cast<const i32x4 *>(p.parts + y * step + 4 * t);
    const f32x4 c = to_float(v) * (p.alpha * p.sx[row]) * scales4(p.sw, col, p.N);
    by_result(p.dtype_c, [&](auto f16, auto out16) {
        store4<decltype(f16)::value, decltype(out16)::value>(p.C + row * p.ldc * (decltype(out16)::value ? 2 : 4), col, p.N, p.beta, c);
    });
}

// Few rows: MB blocks of 16 rows of X by NB blocks of 16 rows of W per
// workgroup, whose eight waves take shares of K of their own (so no wave waits
// for another's loads, and nothing passes through LDS but the sums at the end).
// A lane's 16 bytes of a row are its operand of one v_mfma_i32_16x16x64_i8 as
// they lie in memory; two steps read a row's 128-byte line, and AHEAD lines of
// every row are in flight.
template <int MB, int NB>
__global__ void __launch_bounds__(512) i8_rows_kernel(I8Args p) {
    constexpr int NW = 8, AHEAD = MB + NB <= 3 ? 4 : 2;
    __shared__ i32x4 part[NW][MB * NB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * NB, m0 = blockIdx.y * 16 * MB;
    const char *x[MB], *w[NB];              // (rows past the last: that one again, for outputs that are not stored)
#pragma unroll
    for (int m = 0; m < MB; ++m) x[m] = p.X + min(m0 + 16 * m + lr, p.M - 1) * p.ldx + 16 * lg;
#pragma unroll
    for (int b = 0; b < NB; ++b) w[b] = p.W + min(n0 + 16 * b + lr, p.N - 1) * p.ldw + 16 * lg;
    i32x4 acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = i32x4{0, 0, 0, 0};
    const int lines = (p.K + 127) / 128, last = (int)((long)lines * (wave + 1) / NW);
    const i32x4 none = {0, 0, 0, 0};
    for (int c0 = (int)((long)lines * wave / NW); c0 < last; c0 += AHEAD) {
        i32x4 fx[AHEAD][2][MB], fw[AHEAD][2][NB];
        if ((min(c0 + AHEAD, last)) * 128 <= p.K) {
#pragma unroll
            for (int t = 0; t < AHEAD; ++t) {
                if (t && c0 + t >= last) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = (c0 + t) * 128 + 64 * s;
#pragma unroll
                    for (int b = 0; b < NB; ++b) fw[t][s][b] = *reinterpret_cast<const i32x4 *>(w[b] + k);
#pragma unroll
                    for (int m = 0; m < MB; ++m) fx[t][s][m] = *reinterpret_cast<const i32x4 *>(x[m] + k);
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < AHEAD; ++t) {
                if (t && c0 + t >= last) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = (c0 + t) * 128 + 64 * s, left = p.K - k - 16 * lg;     // integers from this lane's chunk on
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        fw[t][s][b] = none;
                        if (left > 0) fw[t][s][b] = *reinterpret_cast<const i32x4 *>(w[b] + k);
                    }
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        fx[t][s][m] = none;
                        if (left > 0) fx[t][s][m] = *reinterpret_cast<const i32x4 *>(x[m] + k);
                        if (left < 16) fx[t][s][m] = first_bytes(fx[t][s][m], left);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
            if (t && c0 + t >= last) break;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[m][b] = Product<kMulI8>::mfma(fw[t][s][b], fx[t][s][m], acc[m][b]);
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) part[wave][m * NB + b][lane] = acc[m][b];
    __syncthreads();
    // block (m, b)'s lane l holds columns 4*(l/16) .. +3 of row l%16
    for (int t = threadIdx.x; t < MB * NB * 64; t += 64 * NW) {
        const int b = t >> 6, l = t & 63;
        i32x4 v = part[0][b][l];
#pragma unroll
        for (int i = 1; i < NW; ++i) v += part[i][b][l];
        const int row = m0 + 16 * (b / NB) + (l & 15), col = n0 + 16 * (b % NB) + 4 * (l >> 4);
        if (row >= p.M || col >= p.N) continue;
        const f32x4 c = to_float(v) * (p.alpha * p.sx[row]) * scales4(p.sw, col, p.N);
        by_result(p.dtype_c, [&](auto f16, auto out16) {
            store4<decltype(f16)::value, decltype(out16)::value>(p.C + row * p.ldc * (decltype(out16)::value ? 2 : 4), col, p.N, p.beta, c);
        });
    }
}

// ---------------------------------------------------------------------------
// A matrix in 8 bits and back.

struct QuantArgs {
    const char *X;
    signed char *values;
    float *scales;
    char *out;
    long ldx, ldv;
    int M, K;
};

// Eight values of a row from element k on, those from K on 0.
template <int DTYPE>
__device__ __forceinline__ void load8(const char *row, int k, int K, float (&v)[8]) {
    if constexpr (DTYPE == SGEMM_DTYPE_F32) {
        const float *at = reinterpret_cast<const float *>(row) + k;
        if (k + 8 <= K) __builtin_memcpy(v, at, 32);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k + e < K ? at[e] : 0.f;
        }
    } else {
        const unsigned short *at = reinterpret_cast<const unsigned short *>(row) + k;
        unsigned short h[8];
        if (k + 8 <= K) __builtin_memcpy(h, at, 16);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = k + e < K ? at[e] : (unsigned short)0;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = widen16<DTYPE == SGEMM_DTYPE_F16>(h[e]);
    }
}

// x / s to the nearest integer, halves to even, s >= 2^-126.  x * (1 / s) is
// within 2^-16 of the quotient (two roundings of a value of 128 at most), so its
// rounding is right unless it lies that near to a half; then the remainder
// x - q * s, which FP32 holds exactly (a multiple of s's last bit or of x's,
// below 2^24 of them), is compared with half a step.
__device__ __forceinline__ int nearest(float x, float s, float inverse) {
    const float y = x * inverse;
    float q = rintf(y);
    if (fabsf(fabsf(y - q) - 0.5f) < 0x1p-12f) {
        const float rest = __builtin_fmaf(-q, s, x), half = 0.5f * s;
        if (fabsf(rest) > half) q += rest > 0.f ? 1.f : -1.f;
        else if (fabsf(rest) == half && ((int)q & 1)) q += rest > 0.f ? 1.f : -1.f;
    }
    return (int)q;
}

// A row per NT threads, 8 values to a thread and step, PIECES steps of them in
// registers; longer rows are read again (from the cache).  The largest
// magnitude is taken as bits: NaN lies above infinity there, and either makes
// the scale NaN.
template <int DTYPE, int NT>
__global__ void __launch_bounds__(256) i8_quantize_kernel(QuantArgs p) {
    constexpr int PIECES = 2, ROWS = 256 / NT, E = DTYPE == SGEMM_DTYPE_F32 ? 4 : 2;
    __shared__ unsigned tops[4];
    const int t = threadIdx.x % NT;
    const long row = (long)blockIdx.x * ROWS + threadIdx.x / NT;
    const bool live = row < p.M;
    const char *x = p.X + (live ? row : 0) * p.ldx * E;
    float v[PIECES][8];
    unsigned top = 0;
    auto larger = [&](const float (&u)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(u[e]) & 0x7fffffffu);
    };
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        load8<DTYPE>(x, 8 * (t + i * NT), p.K, v[i]);
        larger(v[i]);
    }
    for (int k = 8 * (t + PIECES * NT); k < p.K; k += 8 * NT) {
        float u[8];
        load8<DTYPE>(x, k, p.K, u);
        larger(u);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, d));
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    }
    if (!live) return;
    const bool finite = top < 0x7f800000u;
    const float s = finite ? fmaxf(__fdiv_rn(__uint_as_float(top), 127.f), 0x1p-126f) : __builtin_nanf("");
    const float inverse = __fdiv_rn(1.f, s);
    if (t == 0) p.scales[row] = s;
    signed char *out = p.values + row * p.ldv;
    auto write = [&](const float (&u)[8], int k) {
        if (k >= p.K) return;
        unsigned b[2] = {0, 0};
        if (finite) {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e >> 2] |= (unsigned)(nearest(u[e], s, inverse) & 255) << (8 * (e & 3));
        }
        if (k + 8 <= p.K) __builtin_memcpy(out + k, b, 8);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < p.K) out[k + e] = (signed char)(b[e >> 2] >> (8 * (e & 3)));
        }
    };
#pragma unroll
    for (int i = 0; i < PIECES; ++i) write(v[i], 8 * (t + i * NT));
    for (int k = 8 * (t + PIECES * NT); k < p.K; k += 8 * NT) {
        float u[8];
        load8<DTYPE>(x, k, p.K, u);
        write(u, k);
    }
}

template <int DTYPE>
__global__ void __launch_bounds__(256) i8_dequantize_kernel(QuantArgs p) {
    constexpr int E = DTYPE == SGEMM_DTYPE_F32 ? 4 : 2;
    const int pieces = (p.K + 7) / 8;
    const long all = (long)pieces * p.M;
    for (long t = blockIdx.x * 256L + threadIdx.x; t < all; t += gridDim.x * 256L) {
        const long row = t / pieces;
        const int k = 8 * (int)(t - row * pieces);
        const float s = p.scales[row];
        const signed char *at = p.values + row * p.ldv + k;
        signed char q[8];
        if (k + 8 <= p.K) __builtin_memcpy(q, at, 8);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = k + e < p.K ? at[e] : (signed char)0;
        }
        char *to = p.out + row * p.ldx * E;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = (float)q[4 * h + r] * s;
            if (k + 4 * h < p.K) store4<DTYPE == SGEMM_DTYPE_F16, E == 2>(to, k + 4 * h, p.K, 0.f, v);
        }
    }
}

// f(compile-time element type)
template <class F>
hipError_t by_dtype(int dtype, F &&f) {
    return dtype == SGEMM_DTYPE_BF16 ? f(IntC<SGEMM_DTYPE_BF16>{}) : dtype == SGEMM_DTYPE_F16 ? f(IntC<SGEMM_DTYPE_F16>{}) : f(IntC<SGEMM_DTYPE_F32>{});
}

// ---------------------------------------------------------------------------
// Which kernel.

using Tile64 = TileShape<64, 64, 64, 2, 2, 4, false>;

enum Form { kRows16x16, kRows16x32, kRows32x32, kRows48x32, kRows64x16, kRows64x32, kTile64, kTile128, kTileMixed, kForms };

Form select_form(int M, int N, int K) {
    (void)K;
    const long n32 = (N + 31L) / 32;
    if (M <= 16) return n32 >= 200 ? kRows16x32 : kRows16x16;
    if (M <= 32) return kRows32x32;
    if (M <= 48) return kRows48x32;
    if (M <= 64) return n32 >= 200 ? kRows64x32 : kRows64x16;
    const long t64 = (M + 63L) / 64 * ((N + 63L) / 64), t128 = (M + 127L) / 128 * ((N + 127L) / 128);
    return t64 <= 512 ? kTile64 : t128 <= 512 ? kTile128 : kTileMixed;
}

int select_shares(int, int, int) { return 1; }

template <int MB, int NB>
hipError_t launch_rows8(const I8Args &p, hipStream_t s) {
    return launch_k(i8_rows_kernel<MB, NB>, dim3((unsigned)((p.N + 16 * NB - 1L) / (16 * NB)), (unsigned)((p.M + 16 * MB - 1) / (16 * MB))), dim3(512), s, p);
}

template <class T>
hipError_t launch_tiles(const I8Args &p, int shares, hipStream_t s) {
    const dim3 grid((unsigned)most_tiles(p.groups, p.M, p.N, T::BM, T::BN), (unsigned)shares), block(T::NT);
    if (shares == 1) return launch_k(i8_tile_kernel<T>, grid, block, s, p);
    const hipError_t e = launch_k(i8_share_kernel<T>, grid, block, s, p);
    if (e != hipSuccess) return e;
    return launch_k(i8_join_kernel, dim3((unsigned)(((p.N + 3L) / 4 * p.M + 255) / 256)), dim3(256), s, p, shares);
}

hipError_t launch_mixed(const I8Args &p, hipStream_t s) {
    return launch_k(i8_mixed_kernel, dim3((unsigned)mixed_grid(most_tiles(p.groups, p.M, p.N, 256, 256))), dim3(512), s, p);
}

hipError_t launch_dense(const I8Args &p, int shares, hipStream_t s) {
    switch (select_form(p.M, p.N, p.K)) {
        case kRows16x16: return launch_rows8<1, 1>(p, s);
        case kRows16x32: return launch_rows8<1, 2>(p, s);
        case kRows32x32: return launch_rows8<2, 2>(p, s);
        case kRows48x32: return launch_rows8<3, 2>(p, s);
        case kRows64x16: return launch_rows8<4, 1>(p, s);
        case kRows64x32: return launch_rows8<4, 2>(p, s);
        case kTile64: return launch_tiles<Tile64>(p, shares, s);
        case kTile128: return launch_tiles<Tile128>(p, shares, s);
        default: return launch_mixed(p, s);
    }
}

// Whether one launch can cover the outputs.
bool dense_fits(int M, int N, int K) {
    switch (select_form(M, N, K)) {
        case kTile64: return launch_fits(most_tiles(1, M, N, 64, 64), Tile64::NT);
        case kTile128: return launch_fits(most_tiles(1, M, N, 128, 128), Tile128::NT);
        case kTileMixed: return launch_fits(mixed_grid(most_tiles(1, M, N, 256, 256)), 512);
        default: return launch_fits((N + 15L) / 16, 512);
    }
}

// By the rows of an average group, as the 16-bit products.
hipError_t launch_grouped(const I8Args &p, hipStream_t s) {
    const int rows = p.M / std::min(p.groups, p.M);
    return rows <= 32 ? launch_tiles<Tile32>(p, 1, s) : rows <= 128 ? launch_tiles<Tile128>(p, 1, s) : launch_mixed(p, s);
}

bool grouped_fits(int groups, int M, int N) {
    const int rows = groups > 0 && M > 0 ? M / std::min(groups, M) : 0;
    return rows <= 32    ? launch_fits(most_tiles(groups, M, N, 32, 128), Tile32::NT)
           : rows <= 128 ? launch_fits(most_tiles(groups, M, N, 128, 128), Tile128::NT)
                         : launch_fits(mixed_grid(most_tiles(groups, M, N, 256, 256)), 512);
}

constexpr int kMaxK8 = (1 << 17) - 1;       // sums of products of -128 fit 32 bits
constexpr long kMaxLd8 = 2L * kMaxLd16;
constexpr int kMaxGroups8 = 65535;          // launch grid extent of the padded copies

// Rows of whole aligned chunks; what lies behind K in the last is not used.
bool chunk_rows8(const void *p, long ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 16 == 0 && ld <= kMaxLd8; }

bool dtype_ok(int d) { return d == SGEMM_DTYPE_BF16 || d == SGEMM_DTYPE_F16 || d == SGEMM_DTYPE_F32; }

long copy_bytes(const void *p, long ld, long copies, long stride, long rows, int K) {
    return chunk_rows8(p, ld) && (copies <= 1 || stride % 16 == 0) ? 0 : copies * rows * ceil_to(K, 16);
}

struct Needs {
    long x, w, parts;
    long all() const { return x + w + parts; }
};

Needs i8_needs(int groups, int M, int N, int K, const void *X, int ldx, const void *W, int ldw, long long stride_w, int shares) {
    if (groups == 0 || M == 0 || N == 0 || K == 0) return {0, 0, 0};
    return {ceil_to(copy_bytes(X, ldx, 1, 0, M, K), 256), ceil_to(copy_bytes(W, ldw, groups, stride_w, N, K), 256),
            shares > 1 ? 4L * shares * M * ceil_to(N, 4) : 0};
}

// One 16-byte chunk of dst per thread and step, from rows of any alignment.
__global__ void __launch_bounds__(256) pad_bytes_kernel(const char *src, long ld, long stride, int rows, int cols, char *dst, int chunks) {
    src += blockIdx.y * stride;
    dst += (long)blockIdx.y * rows * chunks * 16;
    const long all = (long)rows * chunks;
    for (long t = blockIdx.x * 256L + threadIdx.x; t < all; t += gridDim.x * 256L) {
        const long r = t / chunks;
        const int c = 16 * (int)(t - r * chunks);
        const char *from = src + r * ld + c;
        i32x4 v = {0, 0, 0, 0};
        if (c + 16 <= cols) {
            __builtin_memcpy(&v, from, 16);
        } else {
            for (int e = 0; c + e < cols; ++e) v[e >> 2] |= (int)((unsigned)(unsigned char)from[e] << (8 * (e & 3)));
        }
        reinterpret_cast<i32x4 *>(dst)[t] = v;
    }
}

hipError_t pad_bytes(const void *src, long ld, long stride, int copies, int rows, int cols, void *dst, hipStream_t s) {
    const int chunks = (cols + 15) / 16;
    return launch_k(pad_bytes_kernel, dim3((unsigned)std::min(((long)rows * chunks + 255) / 256, 1L << 16), (unsigned)copies), dim3(256), s,
                    static_cast<const char *>(src), ld, stride, rows, cols, static_cast<char *>(dst), chunks);
}

// The copies that the operands need, made in the workspace.
hipError_t take_operands(I8Args &p, const Needs &need, char *w, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (need.x) {
        e = pad_bytes(p.X, p.ldx, 0, 1, p.M, p.K, w, s);
        p.X = w;
        p.ldx = ceil_to(p.K, 16);
    }
    if (e == hipSuccess && need.w) {
        e = pad_bytes(p.W, p.ldw, p.strideW, p.groups, p.N, p.K, w + need.x, s);
        p.W = w + need.x;
        p.ldw = ceil_to(p.K, 16);
        p.strideW = p.N * p.ldw;
    }
    p.parts = reinterpret_cast<int *>(w + need.x + need.w);
    return e;
}

bool workspace_ok(long need, const void *workspace, long long bytes) {
    return need == 0 || (workspace != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(workspace) & 15) == 0);
}

constexpr int kWaveRow = 1024;              // longest row that a wave quantises (in registers; a workgroup holds 4096)
constexpr int kMaxRows8 = 1 << 24;          // launch grid extents

int check_quant(int dtype, int M, int K, int ldv, int ldx) {
    if (!dtype_ok(dtype)) return SGEMM_STATUS_INVALID_DTYPE;
    return M < 0 || K < 0 || ldx < std::max(K, 1) || ldv < std::max(K, 1) ? SGEMM_STATUS_INVALID_DIM : SGEMM_STATUS_OK;
}

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

long long sgemm_i8_workspace(int M, int N, int K, const void *X, int ldx, const void *W, int ldw) {
    if (M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    return i8_needs(1, M, N, K, X, ldx, W, ldw, 0, select_shares(M, N, K)).all();
}

int sgemm_i8(int M, int N, int K, float alpha, const void *X, int ldx, const float *x_scales, const void *W, int ldw,
             const float *w_scales, float beta, void *C, int ldc, int dtype_c, void *workspace, long long workspace_bytes,
             void *stream) {
    if (!dtype_ok(dtype_c)) return SGEMM_STATUS_INVALID_DTYPE;
    if (M < 0 || M > kMaxRows8 || N < 0 || N > (1 << 30) || K < 0 || K > kMaxK8) return SGEMM_STATUS_INVALID_DIM;
    if (ldx < std::max(K, 1) || ldw < std::max(K, 1) || ldc < std::max(N, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (!dense_fits(M, N, K)) return SGEMM_STATUS_INVALID_DIM;
    if (M == 0 || N == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || x_scales == nullptr || w_scales == nullptr || (K > 0 && (X == nullptr || W == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    const int shares = select_shares(M, N, K);
    const Needs need = i8_needs(1, M, N, K, X, ldx, W, ldw, 0, shares);
    if (!workspace_ok(need.all(), workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    I8Args p = {static_cast<const char *>(X), static_cast<const char *>(W), x_scales, w_scales, static_cast<char *>(C),
                ldx, ldw, ldc, 0, 0, nullptr, 1, M, N, K, alpha, beta, dtype_c, nullptr};
    hipError_t e = take_operands(p, need, static_cast<char *>(workspace), s);
    if (e == hipSuccess) e = launch_dense(p, shares, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

long long sgemm_i8_grouped_workspace(int groups, int M, int N, int K, const void *X, int ldx, const void *W, int ldw,
                                     long long stride_w) {
    if (groups < 0 || M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    return i8_needs(groups, M, N, K, X, ldx, W, ldw, stride_w, 1).all();
}

int sgemm_i8_grouped(int groups, int M, int N, int K, float alpha, const void *X, int ldx, const float *x_scales,
                     const void *W, int ldw, long long stride_w, const float *w_scales, long long stride_s,
                     const int *offsets, float beta, void *C, int ldc, int dtype_c, void *workspace,
                     long long workspace_bytes, void *stream) {
    if (!dtype_ok(dtype_c)) return SGEMM_STATUS_INVALID_DTYPE;
    if (groups < 0 || groups > kMaxGroups8 || M < 0 || N < 0 || N > kMaxLd16 || K < 0 || K > kMaxK8) return SGEMM_STATUS_INVALID_DIM;
    if (ldx < std::max(K, 1) || ldw < std::max(K, 1) || ldc < std::max(N, 1) || stride_w < 0 || stride_s < 0) return SGEMM_STATUS_INVALID_DIM;
    if (!grouped_fits(groups, M, N)) return SGEMM_STATUS_INVALID_DIM;
    if (groups == 0 || M == 0 || N == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || offsets == nullptr || x_scales == nullptr || w_scales == nullptr || (K > 0 && (X == nullptr || W == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    const Needs need = i8_needs(groups, M, N, K, X, ldx, W, ldw, stride_w, 1);
    if (!workspace_ok(need.all(), workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    I8Args p = {static_cast<const char *>(X), static_cast<const char *>(W), x_scales, w_scales, static_cast<char *>(C),
                ldx, ldw, ldc, stride_w, stride_s, offsets, groups, M, N, K, alpha, beta, dtype_c, nullptr};
    hipError_t e = take_operands(p, need, static_cast<char *>(workspace), s);
    if (e == hipSuccess) e = launch_grouped(p, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_i8_quantize(int dtype, int M, int K, const void *X, int ldx, void *values, int ldv, float *scales, void *stream) {
    const int st = check_quant(dtype, M, K, ldv, ldx);
    if (st != SGEMM_STATUS_OK) return st;
    if (!launch_fits(K <= kWaveRow ? (M + 3L) / 4 : M, 256)) return SGEMM_STATUS_INVALID_DIM;
    if (M == 0) return SGEMM_STATUS_OK;
    if (scales == nullptr || (K > 0 && (X == nullptr || values == nullptr))) return SGEMM_STATUS_NULL_POINTER;
    const QuantArgs p = {static_cast<const char *>(X), static_cast<signed char *>(values), scales, nullptr, ldx, ldv, M, K};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = by_dtype(dtype, [&](auto d) {
        constexpr int D = decltype(d)::value;
        return p.K <= kWaveRow ? launch_k(i8_quantize_kernel<D, 64>, dim3((unsigned)((p.M + 3L) / 4)), dim3(256), s, p)
                           : launch_k(i8_quantize_kernel<D, 256>, dim3((unsigned)p.M), dim3(256), s, p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_i8_dequantize(int dtype, int M, int K, const void *values, int ldv, const float *scales, void *X, int ldx, void *stream) {
    const int st = check_quant(dtype, M, K, ldv, ldx);
    if (st != SGEMM_STATUS_OK) return st;
    if (M == 0 || K == 0) return SGEMM_STATUS_OK;
    if (scales == nullptr || X == nullptr || values == nullptr) return SGEMM_STATUS_NULL_POINTER;
    const QuantArgs p = {nullptr, static_cast<signed char *>(const_cast<void *>(values)), const_cast<float *>(scales), static_cast<char *>(X), ldx, ldv, M, K};
    const hipError_t e = by_dtype(dtype, [&](auto d) {
        return launch_k(i8_dequantize_kernel<decltype(d)::value>, dim3((unsigned)std::min(((p.K + 7L) / 8 * p.M + 255) / 256, 1L << 16)), dim3(256),
                        reinterpret_cast<hipStream_t>(stream), p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

}  // extern "C"

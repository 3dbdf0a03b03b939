// What the kernels built on the 16-bit K loop (sgemm_lowp.hpp) share beyond
// it: tile shapes, the raster of a tile grid whose height only the device
// knows, and stores of FP32 accumulators as FP32 or 16-bit values.
#pragma once

#include "../../include/sgemm.h"
#include "sgemm_lowp.hpp"

namespace sgemm_mi355x {

// Status of a HIP error for the C ABI, its text kept for
// sgemm_last_hip_error() (defined with the other entry points).
int hip_status(hipError_t e, const char *what);

// A block tile: BM x BN outputs, BK-deep K tiles, WM x WN waves, NS stages,
// PP the alternating schedule (see lowp_accumulate).
template <int BM_, int BN_, int BK_, int WM_, int WN_, int NS_, bool PP_>
struct TileShape {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WAVES_M = WM_, WAVES_N = WN_, NS = NS_;
    static constexpr bool PP = PP_;
    static constexpr int NT = 64 * WM_ * WN_;
    static constexpr int WM = BM_ / WM_, WN = BN_ / WN_;       // outputs per wave
    static constexpr int MI = WM / 16, NB = WN / 16;           // 16x16 blocks per wave
    static constexpr int LDS = NS_ * (BM_ + BN_) * BK_ * 2;
};
using Tile32 = TileShape<32, 128, 64, 1, 4, 4, false>;
using Tile128 = TileShape<128, 128, 64, 2, 2, 2, false>;     // two workgroups to a compute unit
using TileWide = TileShape<128, 256, 32, 2, 4, 3, true>;
using TileTall = TileShape<256, 128, 64, 2, 4, 3, false>;
using TileQuarter = TileShape<128, 128, 64, 2, 4, 4, true>;
using Tile256 = TileShape<256, 256, 32, 2, 4, 4, true>;

// The operands of one tile's product as lowp_accumulate takes them.
struct Operands16 {
    const char *A, *B;
    long lda, ldb;
    int M, N, K;
};

template <class T, bool F16, bool TA, bool TB>
__device__ __forceinline__ void accumulate16(const Operands16 &q, int m0, int n0, char *lds, f32x4 (&acc)[T::MI][T::NB]) {
    lowp_accumulate<T::BM, T::BN, T::BK, T::WAVES_M, T::WAVES_N, T::NS, T::PP, true, F16, false, TA, TB>(
        q, m0, n0, lds, 1, 0, acc);
}

// Workgroup `bid` of `total`: each of the 8 XCDs, which take workgroups in
// turn, gets a contiguous run of tiles, so that tiles that share operands
// share an L2.  A permutation of 0 .. total - 1.
__device__ __forceinline__ int xcd_run(int bid, int total) {
    const int per = total >> 3;
    return bid < (per << 3) ? (bid & 7) * per + (bid >> 3) : bid;
}

// Tile number `id` of a tiles_m x tiles_n grid, in runs of up to eight tile
// rows by all tile columns, so that the tiles in flight on an XCD form a
// compact patch.
__device__ __forceinline__ void raster(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
    constexpr int GM = 8;
    const int g = id / (GM * tiles_n), in = id - g * GM * tiles_n;
    const int rows = min(tiles_m - g * GM, GM);
    tm = g * GM + in % rows;
    tn = in / rows;
}

// A grid of `total` tiles of 256 x 256 over the 256 compute units, one
// workgroup each: whole rounds run on Tile256, and a last round that fills at
// most half of the chip is cut finer, in two (TileWide, or with B transposed
// TileTall) or, below a quarter, in four, so that its tiles take 0.57 or 0.39
// of a round instead of a whole one.  16384 rows in 16 even groups, BF16: 4096
// columns by 2048 k 282 us on Tile256 alone, 288 on TileWide alone, 259 so; B
// transposed, 2048 by 4096, 295, 280 (TileTall) and 250 (uneven groups, as a
// router fills them, take 297 and 300: more partly filled tiles); but 3001 rows in
// 5 groups by 5000 by 2048, just over one round, 89, 63 and 72.
// body.tile<T>(lds, id, sub) does part `sub` of tile number `id`; the number of
// tiles need only be known here.  Launched with mixed_grid(largest total)
// workgroups of 512 threads.
template <bool TB>
struct Mixed {
    using Half = typename std::conditional<TB, TileTall, TileWide>::type;
    static constexpr int NT = 512;
    static constexpr int LDS = Half::LDS > Tile256::LDS ? Half::LDS : Tile256::LDS;
    static_assert(Tile256::NT == NT && Half::NT == NT && TileQuarter::NT == NT && TileQuarter::LDS <= LDS, "one launch");
    template <class Body>
    static __device__ __forceinline__ void run(const Body &body, char *lds, int total) {
        const int bid = blockIdx.x, whole = total & ~255, rest = total - whole, k = bid - whole;
        if (k < 0) body.template tile<Tile256>(lds, xcd_run(bid, whole), 0);
        else if (rest > 128) {
            if (k < rest) body.template tile<Tile256>(lds, whole + xcd_run(k, rest), 0);
        } else if (rest > 64) {
            if (k >= 2 * rest) return;
            const int at = xcd_run(k, 2 * rest);
            body.template tile<Half>(lds, whole + (at >> 1), at & 1);
        } else if (k < 4 * rest) {
            const int at = xcd_run(k, 4 * rest);
            body.template tile<TileQuarter>(lds, whole + (at >> 2), at & 3);
        }
    }
};

constexpr long mixed_grid(long total) { return total + 256; }   // (whole rounds, and 256 at most behind them)

// Corner of part `sub` of the 256 x 256 tile (tm, tn) for tile T.
template <class T>
__device__ __forceinline__ void part_corner(int tm, int tn, int sub, int &m0, int &n0) {
    constexpr int PN = 256 / T::BN;
    m0 = tm * 256 + sub / PN * T::BM;
    n0 = tn * 256 + sub % PN * T::BN;
}

// Four FP32 values rounded to 16 bits (to nearest, ties to even).
template <bool F16>
__device__ __forceinline__ i32x2 round16(f32x4 v) {
    if constexpr (F16) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(i32x2, __builtin_convertvector(v, h4));
    } else {
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(i32x2, __builtin_convertvector(v, b4));
    }
}

template <bool F16>
__device__ __forceinline__ float widen16(unsigned short bits) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, bits);
    return __uint_as_float((unsigned)bits << 16);
}

// Columns col .. col+3 (those below N) of a row of C at `row`, C of FP32 or
// (OUT16) 16-bit values: v, plus beta times what is there unless beta is 0
// (then C is not read).  The four go in one access whatever the row's
// alignment: this chip takes such accesses at any element.
template <bool F16, bool OUT16>
__device__ __forceinline__ void store4(char *row, int col, int N, float beta, f32x4 v) {
    if constexpr (OUT16) {
        unsigned short *dst = reinterpret_cast<unsigned short *>(row) + col;
        if (beta != 0.f) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (col + r < N) v[r] += beta * widen16<F16>(dst[r]);
        }
        const i32x2 o = round16<F16>(v);
        if (col + 3 < N) {
            __builtin_memcpy(dst, &o, 8);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (col + r < N) dst[r] = (unsigned short)((unsigned)o[r >> 1] >> (16 * (r & 1)));
        }
    } else {
        float *dst = reinterpret_cast<float *>(row) + col;
        if (col + 3 < N) {
            if (beta != 0.f) {
                f32x4 c;
                __builtin_memcpy(&c, dst, 16);
                v += c * beta;
            }
            __builtin_memcpy(dst, &v, 16);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (col + r < N) dst[r] = v[r] + (beta != 0.f ? beta * dst[r] : 0.f);
        }
    }
}

// C[rows below M][columns below N] = alpha * acc + beta * C for the tile at
// (m0, n0): block (mi, nb) of a lane holds row l%16 and columns 4*(l/16)..+3.
template <class T, bool F16, bool OUT16>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[T::MI][T::NB], int m0, int n0, int M, int N, char *C,
                                           long ldc, float alpha, float beta) {
    constexpr int E = OUT16 ? 2 : 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
        const int row = m0 + (wave / T::WAVES_N) * T::WM + mi * 16 + (lane & 15);
        if (row >= M) continue;
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) {
            const int col = n0 + (wave % T::WAVES_N) * T::WN + nb * 16 + 4 * (lane >> 4);
            store4<F16, OUT16>(C + (long)row * ldc * E, col, N, beta, acc[mi][nb] * alpha);
        }
    }
}

// The sum of `shares` groups of four values `step` floats apart, in order, with
// sixteen loads in flight.
__device__ __forceinline__ f32x4 sum_shares(const float *at, long step, int shares) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int y = 0; y < shares; y += 16) {
        f32x4 x[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) x[u] = *reinterpret_cast<const f32x4 *>(at + min(y + u, shares - 1) * step);
#pragma unroll
        for (int u = 0; u < 16; ++u)
            if (y + u < shares) v += x[u];
    }
    return v;
}

inline long ceil_to(long n, long to) { return (n + to - 1) / to * to; }

// Largest leading dimension of the 16-bit kernels' operands: 256 rows of a K
// tile, or with the operand transposed the K tile's 64 of 256 columns, stay
// within the 31-bit range of a buffer descriptor, so that kOutOfRange lies
// behind it.
constexpr int kMaxLd16 = (1 << 22) - 64;
static_assert(2L * (255L * kMaxLd16 + 64) <= kOutOfRange && 2L * (63L * kMaxLd16 + 256) <= kOutOfRange, "descriptor range");

// Whether one launch can have that many workgroups of `threads` (HIP takes
// fewer than 2^32 threads).
inline bool launch_fits(long workgroups, int threads) { return workgroups <= 0xffffffffL / threads; }

inline bool chunk_rows(const void *p, long ld, long cols) {     // rows of whole 16-byte chunks
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && cols % 8 == 0 && ld <= kMaxLd16;
}

// dst [copies][rows][cols8] = src [copies][rows][cols] (row length cols8:
// cols rounded up to whole 16-byte chunks, zeros behind cols); up to 65535
// copies.
hipError_t pad_rows(const void *src, long ld, long stride, int copies, int rows, int cols, void *dst, hipStream_t s);

}  // namespace sgemm_mi355x

// GEMM with BF16 or FP16 inputs and FP32 accumulation and output:
// C = alpha * A * B + beta * C, A [M,K] and B [K,N] row-major 16-bit, C
// [M,N] row-major FP32.  (Built with MFMA results in VGPRs; see
// sgemm_lean.hpp.)  The K loop and its layouts are in sgemm_lowp.hpp; this
// unit adds the split-K hand-off and the epilogue.
#include "sgemm_lowp.hpp"

namespace sgemm_mi355x {

template <int BM, int BN, int BK, int WAVES_M, int WAVES_N, int NSTAGE, bool PP, bool BETA0, bool EDGE, bool F16,
          bool SPLIT, bool TA = false, bool TB = false>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N)
sgemm_lowp_kernel(Args p) {
    constexpr int NT = 64 * WAVES_M * WAVES_N;
    constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    constexpr int MI = WM / 16, NB = WN / 16;               // 16x16 blocks per wave
    __shared__ __attribute__((aligned(16))) char lds[NSTAGE * (BM + BN) * BK * 2];

    batch_offset<2>(p);                                     // problem blockIdx.z of a strided batch
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int lrow = tid & 15, lg = (tid & 63) >> 4;
    int tm, tn;
    const int slot = tile_coords(p, tm, tn);          // split-K workspace slot
    const int m0 = tm * BM, n0 = tn * BN;
    f32x4 acc[MI][NB];
    lowp_accumulate<BM, BN, BK, WAVES_M, WAVES_N, NSTAGE, PP, EDGE, F16, SPLIT, TA, TB>(
        p, m0, n0, lds, SPLIT ? gridDim.y : 1, SPLIT ? blockIdx.y : 0, acc);

    if constexpr (SPLIT) {
        if (!split_reduce_n<NT, MI * NB>(p, slot, tid, reinterpret_cast<unsigned *>(lds),
                                         [&](int c) -> f32x4 & { return acc[c / NB][c % NB]; }))
            return;
    }

    // C = alpha * acc (+ beta * C): block (mi, nb) holds row l%16 and
    // columns 4*(l/16) .. +3 of its 16x16 output block; 16-byte accesses
    // when C's rows are 16-byte aligned and the four columns lie below N.
    // (N need not be a multiple of 4: the product on the library's padded
    // copies runs with the true N, so the last vector of a row may straddle
    // N; its columns are then stored one by one.)
    const float alpha = p.alpha, beta = p.beta;
    const bool vecc = (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 && (p.ldc & 3) == 0;
    if constexpr (BETA0 || EDGE) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int row = m0 + wm * WM + mi * 16 + lrow;
                const int col = n0 + wn * WN + nb * 16 + 4 * lg;
                if (EDGE && row >= p.M) continue;
                float *dst = p.C + (long)row * p.ldc + col;
                if (vecc && (!EDGE || col + 3 < p.N)) {
                    f32x4 o = acc[mi][nb] * alpha;
                    if (!BETA0) o += *reinterpret_cast<const f32x4 *>(dst) * beta;
                    *reinterpret_cast<f32x4 *>(dst) = o;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (EDGE && col + r >= p.N) continue;
                        float o = alpha * acc[mi][nb][r];
                        if (!BETA0) o += beta * dst[r];
                        dst[r] = o;
                    }
                }
            }
        return;
    }
    // Whole tiles with beta != 0: the C values of a row group's NB blocks
    // are loaded before the first of their stores.  Each is read and written
    // by this lane alone and the rows of C are disjoint (ldc >= N), so the
    // order is free, and the loads wait for memory once per row group
    // instead of once per block (a compiler cannot move a load above a store
    // it cannot prove disjoint).  The 16-byte test of C is taken once,
    // outside the loops, so that no branch splits a row group's loads from
    // its stores.  (4096^3 BF16, alpha = beta = 1: 117.7 -> 112.3 us.  Edge
    // tiles keep the per-block order: their guarded loads, made branch-free,
    // ran slower than the waits they saved.)
    auto write = [&](auto vec_c) __attribute__((always_inline)) {
        constexpr bool VC = decltype(vec_c)::value;
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
            const int row = m0 + wm * WM + mi * 16 + lrow;
            f32x4 cin[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float *src = p.C + (long)row * p.ldc + n0 + wn * WN + nb * 16 + 4 * lg;
                if constexpr (VC) {
                    cin[nb] = *reinterpret_cast<const f32x4 *>(src);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) cin[nb][r] = src[r];
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float *dst = p.C + (long)row * p.ldc + n0 + wn * WN + nb * 16 + 4 * lg;
                if constexpr (VC) {
                    *reinterpret_cast<f32x4 *>(dst) = acc[mi][nb] * alpha + cin[nb] * beta;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) dst[r] = alpha * acc[mi][nb][r] + beta * cin[nb][r];
                }
            }
        }
    };
    if (vecc) write(std::true_type{});
    else write(std::false_type{});
}

template <int BM, int BN, int BK, int WM, int WN, int NSTAGE, bool F16, bool PP, bool SPLIT, bool TA = false,
          bool TB = false>
hipError_t launch_lowp(const Args &a0, hipStream_t stream, int batch = 1) {
    const Args a = tiled(a0, BM, BN);
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n), (unsigned)(SPLIT ? a.splits : 1), (unsigned)batch);
    const dim3 block(64 * WM * WN);
    const bool edge = (a.M % BM) || (a.N % BN) || (a.K % BK);
#define SGEMM_LAUNCH(Z, E) \
    launch_k(sgemm_lowp_kernel<BM, BN, BK, WM, WN, NSTAGE, PP, Z, E, F16, SPLIT, TA, TB>, grid, block, stream, a)
    if (edge) {
        if (a.beta == 0.0f) return SGEMM_LAUNCH(true, true);
        return SGEMM_LAUNCH(false, true);
    }
    if (a.beta == 0.0f) return SGEMM_LAUNCH(true, false);
    return SGEMM_LAUNCH(false, false);
#undef SGEMM_LAUNCH
}

// One alternating kernel with each of the four operand orientations (SP:
// its split-K form).
template <int BM, int BN, int BK, int NS, bool SP>
hipError_t launch_lowp_alt_op(const Args &a, bool f16, bool ta, bool tb, int batch, hipStream_t s) {
#define SGEMM_O(F, A, B) launch_lowp<BM, BN, BK, 2, 4, NS, F, true, SP, A, B>(a, s, batch)
    if (f16) {
        if (ta && tb) return SGEMM_O(true, true, true);
        if (ta) return SGEMM_O(true, true, false);
        if (tb) return SGEMM_O(true, false, true);
        return SGEMM_O(true, false, false);
    }
    if (ta && tb) return SGEMM_O(false, true, true);
    if (ta) return SGEMM_O(false, true, false);
    if (tb) return SGEMM_O(false, false, true);
    return SGEMM_O(false, false, false);
#undef SGEMM_O
}

// Launcher called from the C ABI's translation unit; `tile` picks the block
// tile, K tile, waves and number of stages (the table of variants in the C
// ABI's translation unit lists them in this order).  a.splits > 1 runs the
// split-K form (built for the 128x128 two-stage kernel and the 128x128
// alternating kernel); ta / tb (transposed operands) are built for the two
// alternating kernels; batch problems on gridDim.z.  Returns the launch's
// status.
hipError_t launch_lowp_tile(const Args &a, bool f16, int tile, bool ta, bool tb, int batch, hipStream_t s) {
#define SGEMM_T(BM, BN, BK, WM, WN, NS, PP, SP)                                          \
    (f16 ? launch_lowp<BM, BN, BK, WM, WN, NS, true, PP, SP>(a, s, batch)                \
         : launch_lowp<BM, BN, BK, WM, WN, NS, false, PP, SP>(a, s, batch))
    const bool split = a.splits > 1;
    switch (tile) {
        case 1: return SGEMM_T(256, 128, 64, 2, 4, 3, false, false);
        case 2: return SGEMM_T(256, 256, 32, 2, 4, 4, false, false);
        case 3: return launch_lowp_alt_op<256, 256, 32, 4, false>(a, f16, ta, tb, batch, s);
        case 4:
            if (split) return launch_lowp_alt_op<128, 128, 64, 4, true>(a, f16, ta, tb, batch, s);
            return launch_lowp_alt_op<128, 128, 64, 4, false>(a, f16, ta, tb, batch, s);
        default:
            if (split) return SGEMM_T(128, 128, 64, 2, 2, 2, false, true);
            return SGEMM_T(128, 128, 64, 2, 2, 2, false, false);
    }
#undef SGEMM_T
}

}  // namespace sgemm_mi355x

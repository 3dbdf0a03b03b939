// Products with 4-bit weights: C = alpha * X * W^T + beta * C, X [M,K] and
// (after rounding) C in 16 bits or C in FP32, W [N,K] held as
// w = (q - z) * s with 4-bit q, one scale s (and one zero point z, else 8)
// for each `group` consecutive k of a row; and the kernels that bring a
// 16-bit weight into that form and back.
//
// Packed form.  A row holds K rounded up to whole chunks of 128 k, 64 bytes
// each, as four runs (j = 0..3) of four 32-bit words (s = 0..3); word (j, s)
// holds k = 32 s + 8 j .. + 7 of the chunk, element 2i in bits 4i..4i+3 and
// element 2i + 1 in bits 16+4i..16+4i+3.  So one 16-byte load gives lane
// (n = l%16, j = l/16) its share of four k steps of the matrix instruction
// v_mfma_f32_16x16x32, each step within one group of 32 or more, and each
// word becomes four registers of two neighbouring 16-bit values with a shift
// and an and-or:
//
// A nibble put into the top mantissa bits below the exponent of 16 is the
// 16-bit value 16 + q, exactly, for bf16 (q at bit 3) and fp16 (q at bit 6).
// The instruction then sums x * (16 + q) exactly as it would x * w, a second
// one with a matrix of ones gives the sum of x, and per group
//     sum x * (q - z) * s = s * (sum x * (16 + q) - (16 + z) * sum x)
// in FP32, so the weights are never rounded and the scale costs one
// multiply-add per output and group.  With an infinity in X, or BF16 values
// above 2^128 / 31, the two sums may pass FP32's range where their difference
// does not; what comes out is then infinite or NaN, and such an output is
// formed again from q - z.
#include <algorithm>

#include "sgemm_tile16.hpp"

namespace sgemm_mi355x {

namespace {

constexpr int kChunk = 128;             // k per packed chunk of 64 bytes

struct W4Args {
    const char *X;                      // 16-bit
    const unsigned char *packed, *zeros;
    const unsigned short *scales;       // 16-bit floats of X's type
    char *C;
    long ldx, ldc;
    int M, N, K, chunks;
    float alpha, beta;
};

// The scales of a row's chunk (in one register), those of groups wholly behind
// K taken as 0: they belong to no weight, and a NaN there must not meet the
// zeros that X counts as behind K.  `last`: of the row.
template <int GROUP, class S>
__device__ __forceinline__ S used_scales(S scales, bool last, int K) {
    constexpr int GPC = kChunk / GROUP;
    const int groups = ((K - 1) % kChunk) / GROUP + 1;     // of the last chunk that hold a k (K > 0)
    return last && groups < GPC ? scales & (((S)1 << (16 * groups % (8 * sizeof(S)))) - 1) : scales;
}

// The two 16-bit values 16 + q of nibble i of each half of a word.
template <bool F16, int I>
__device__ __forceinline__ int q_pair(unsigned w) {
    constexpr int to = (F16 ? 6 : 3) - 4 * I;              // shift left
    const unsigned v = to >= 0 ? w << (to >= 0 ? to : 0) : w >> (to < 0 ? -to : 0);
    return (int)((v & (F16 ? 0x03C003C0u : 0x00780078u)) | (F16 ? 0x4C004C00u : 0x41804180u));
}

// sum x * (q - z) * s for one output, a multiplication at a time (for all
// outputs of 64 rows of NaN by 8192 x 4096 1.05 ms in place of 19 us).
template <int GROUP, bool ZEROS, bool F16>
__device__ __forceinline__ float w4_output(const W4Args &p, int row, int col) {
    const unsigned short *x = reinterpret_cast<const unsigned short *>(p.X) + row * p.ldx;
    const unsigned *words = reinterpret_cast<const unsigned *>(p.packed + (long)col * p.chunks * 64);
    const long first = (long)col * p.chunks * (kChunk / GROUP);
    float total = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < p.K; k0 += 8) {
        const unsigned w = words[k0 / kChunk * 16 + k0 % 32 / 8 * 4 + k0 % kChunk / 32];
        const float z = ZEROS ? (float)p.zeros[first + k0 / GROUP] : 8.f;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += widen16<F16>(x[k0 + e]) * ((float)(w >> (4 * (e >> 1) + 16 * (e & 1)) & 15) - z);
        total += sum * widen16<F16>(p.scales[first + k0 / GROUP]);
    }
    return total;
}

// Few rows of X: MB blocks of 16 of them by NB blocks of 16 rows of W per
// workgroup, whose NW waves take consecutive runs of chunks and add up
// through LDS.  The weights' bytes bound it as far as the vector memory path
// of a compute unit keeps up (64 bytes a clock, and a cycle for each 128-byte
// line that a load touches), so that path is spared: a wave loads four chunks
// of weights at once, one load brings the scales of four chunks (lane
// (n, j) has row n's of chunk j; they are handed round in registers), and
// lanes of rows past M load nothing.  GROUP: k per scale.
template <int MB, int NB, int NW, int GROUP, bool ZEROS, bool F16, bool OUT16>
__global__ void __launch_bounds__(64 * NW) w4_rows_kernel(W4Args p) {
    constexpr int GPC = kChunk / GROUP, SPG = 4 / GPC;      // groups per chunk, k steps per group
    using Scales = typename std::conditional<GPC == 4, unsigned long, unsigned>::type;
    __shared__ f32x4 part[NW][MB * NB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * NB, m0 = blockIdx.y * 16 * MB;
    const unsigned char *wtile = p.packed + (long)n0 * p.chunks * 64;
    const unsigned char *ztile = ZEROS ? p.zeros + (long)n0 * p.chunks * GPC : nullptr;
    const unsigned short *stile = p.scales + (long)n0 * p.chunks * GPC;
    const unsigned short *xtile = reinterpret_cast<const unsigned short *>(p.X) + (long)m0 * p.ldx;
    unsigned first[NB], xrow[MB];                           // first chunk of this lane's rows of W; its rows of X
    bool live[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b) first[b] = (unsigned)(min(16 * b + lr, p.N - 1 - n0) * p.chunks);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        live[m] = 16 * m + lr < p.M - m0;
        xrow[m] = (unsigned)(16 * m + lr) * (unsigned)p.ldx + 8 * lg;
    }
    const int one = F16 ? 0x3C003C00 : 0x3F803F80;
    const i32x4 ones = {one, one, one, one};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 total[MB][NB];
    i32x4 x[2][4][MB];                                      // two chunks of X in turn
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
        for (int b = 0; b < NB; ++b) total[m][b] = zero;
#pragma unroll
        for (int s = 0; s < 4; ++s) x[0][s][m] = x[1][s][m] = i32x4{0, 0, 0, 0};
    }
    // (what a lane of a row past M holds only reaches results of such rows)
    auto load_x = [&](int c, i32x4 (&to)[4][MB]) {
        const unsigned short *xc = xtile + (long)c * kChunk;
        const bool whole = (c + 1) * kChunk <= p.K;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (whole) {
                if (live[m]) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) to[s][m] = *reinterpret_cast<const i32x4 *>(xc + (xrow[m] + 32 * s));
                }
            } else {                                        // (K is a multiple of 8 here)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    to[s][m] = i32x4{0, 0, 0, 0};
                    if (live[m] && c * kChunk + 32 * s + 8 * lg < p.K)
                        to[s][m] = *reinterpret_cast<const i32x4 *>(xc + (xrow[m] + 32 * s));
                }
            }
        }
    };
    const int last = (int)((long)p.chunks * (wave + 1) / NW);
    for (int c0 = (int)((long)p.chunks * wave / NW); c0 < last; c0 += 4) {
        i32x4 w[4][NB];
        Scales four_s[NB];
        unsigned four_z[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t == 0 || c0 + t < last)
                    w[t][b] = *reinterpret_cast<const i32x4 *>(wtile + ((first[b] + c0 + t) * 64 + 16 * lg));
            const unsigned at = first[b] + min(c0 + lg, last - 1);
            if constexpr (GPC > 1)
                four_s[b] = used_scales<GROUP>(*reinterpret_cast<const Scales *>(stile + at * GPC), c0 + lg >= p.chunks - 1, p.K);
            else four_s[b] = stile[at];
            if constexpr (ZEROS && GPC == 4) four_z[b] = *reinterpret_cast<const unsigned *>(ztile + at * GPC);
            else if constexpr (ZEROS && GPC == 2) four_z[b] = *reinterpret_cast<const unsigned short *>(ztile + at * GPC);
            else four_z[b] = ZEROS ? ztile[at] : 0x08080808u;
        }
        load_x(c0, x[0]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (c0 + t >= last) break;
            if (t < 3 && c0 + t + 1 < last) load_x(c0 + t + 1, x[(t + 1) & 1]);
            f32x4 sum[MB][NB], sx[MB];
            Scales sc[NB];
            unsigned zp[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                sc[b] = __shfl(four_s[b], 16 * t + lr);
                zp[b] = ZEROS ? __shfl(four_z[b], 16 * t + lr) : 0x08080808u;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    sx[m] = mfma_16x16x32<F16>(x[t & 1][s][m], ones, s % SPG == 0 ? zero : sx[m]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const unsigned v = w[t][b][s];
                    const i32x4 wf = {q_pair<F16, 0>(v), q_pair<F16, 1>(v), q_pair<F16, 2>(v), q_pair<F16, 3>(v)};
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        sum[m][b] = mfma_16x16x32<F16>(x[t & 1][s][m], wf, s % SPG == 0 ? zero : sum[m][b]);
                }
                if (s % SPG == SPG - 1) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float scale = widen16<F16>((unsigned short)(sc[b] >> (16 * (s / SPG))));
                        const float z = 16.f + (float)(zp[b] >> (8 * (s / SPG)) & 255);
#pragma unroll
                        for (int m = 0; m < MB; ++m) total[m][b] += (sum[m][b] - sx[m] * z) * scale;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) part[wave][m * NB + b][lane] = total[m][b];
    __syncthreads();
    // block (m, b)'s lane l holds rows 4*(l/16) .. +3 of column l%16
    for (int t = threadIdx.x; t < MB * NB * 64; t += 64 * NW) {
        const int b = t >> 6, l = t & 63;
        f32x4 v = part[0][b][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w][b][l];
        const int col = n0 + 16 * (b % NB) + (l & 15);
        if (col >= p.N) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = m0 + 16 * (b / NB) + 4 * (l >> 4) + r;
            if (row >= p.M) continue;
            if (!(fabsf(v[r]) < __builtin_inff())) v[r] = w4_output<GROUP, ZEROS, F16>(p, row, col);
            float o = p.alpha * v[r];
            if constexpr (OUT16) {
                unsigned short *dst = reinterpret_cast<unsigned short *>(p.C) + row * p.ldc + col;
                if (p.beta != 0.f) o += p.beta * widen16<F16>(*dst);
                const f32x4 o4 = {o, o, o, o};
                *dst = (unsigned short)round16<F16>(o4)[0];
            } else {
                float *dst = reinterpret_cast<float *>(p.C) + row * p.ldc + col;
                *dst = p.beta != 0.f ? o + p.beta * *dst : o;
            }
        }
    }
}

// The eight values q - z of a word, exactly, as four registers of pairs;
// zs: 16 + z (fp16: twice in 16 bits; bf16: z in FP32).
template <bool F16>
__device__ __forceinline__ i32x4 centred(unsigned w, unsigned zs) {
    if constexpr (F16) {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 z = __builtin_bit_cast(h2, zs);
        return i32x4{__builtin_bit_cast(int, __builtin_bit_cast(h2, q_pair<true, 0>(w)) - z),
                     __builtin_bit_cast(int, __builtin_bit_cast(h2, q_pair<true, 1>(w)) - z),
                     __builtin_bit_cast(int, __builtin_bit_cast(h2, q_pair<true, 2>(w)) - z),
                     __builtin_bit_cast(int, __builtin_bit_cast(h2, q_pair<true, 3>(w)) - z)};
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        typedef float f2 __attribute__((ext_vector_type(2)));
        const float z = __uint_as_float(zs);
        // bytes 0..3 of `even` are nibbles 0, 2, 4, 6, of `odd` 1, 3, 5, 7
        const unsigned even = w & 0x0F0F0F0Fu, odd = w >> 4 & 0x0F0F0F0Fu;
        auto pair = [&](unsigned v, int lo) {
            const f2 f = {(float)(v >> (8 * lo) & 255) - z, (float)(v >> (8 * lo + 16) & 255) - z};
            return __builtin_bit_cast(int, __builtin_convertvector(f, b2));
        };
        return i32x4{pair(even, 0), pair(odd, 0), pair(even, 1), pair(odd, 1)};
    }
}

// Many rows of X: a workgroup of WM x WN waves takes 16*MI*WM rows of X by
// 16*NB*WN rows of W.  X comes through LDS (direct loads of one 128-k chunk,
// two stages, rows of 256 bytes, 16-byte chunk c of row m at c ^ (m % 16): no
// bank conflicts counted); the weights go from memory straight into the registers
// of the one wave that multiplies them, so each is unpacked once per tile and
// only X loads the LDS.  q - z is exact in 16 bits; two k steps of a group
// (one for groups of 32) are summed by the matrix instructions and then added
// to the FP32 total with the group's scale.  Those multiply-adds and the
// unpacking take about as many cycles as the matrix instructions, so every
// matrix instruction is followed by its share of them: left to itself the
// compiler gathers each kind, and the same tile took a ninth longer.  2048 x
// 8192 x 4096, groups of 64 with zero points, FP16: 169 us in a row of calls (813
// TFLOP/s; 183 to 190 us under a kernel trace, matrix instructions 34% of the
// time under counters); two workgroups of four waves share a compute unit (one
// of eight, in step at every barrier, took 170 us where these took 165).  The
// product is formed transposed, as in
// sgemm_lowp.hpp: lane l holds row l%16 and columns 4*(l/16) .. +3.
template <int MI, int NB, int WM, int WN, int GROUP, bool ZEROS, bool F16, bool OUT16>
__global__ void __launch_bounds__(64 * WM * WN, 2) w4_tile_kernel(W4Args p) {
    constexpr int GPC = kChunk / GROUP, SPG = GROUP == 32 ? 1 : 2, PARTS = 4 / SPG;
    constexpr int NWAVES = WM * WN, BM = 16 * MI * WM, BN = 16 * NB * WN;
    constexpr int STAGE = BM * 256, L = STAGE / 16 / (64 * NWAVES);
    __shared__ __attribute__((aligned(16))) char lds[2 * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    raster(xcd_run(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    // direct loads: load i of a wave fills four rows of a stage, 16-byte chunk
    // c8 / 8 of them in this lane (the layout's swizzle, the same for every i)
    const int row0 = 4 * wave + lg, c8 = 8 * (lr ^ (row0 & 15)), rows = min(BM, p.M - m0);
    const unsigned off0 = 2u * (unsigned)(row0 * (int)p.ldx + c8), step = 2u * 4 * NWAVES * (unsigned)p.ldx;
    static_assert(4 * NWAVES % 16 == 0, "one swizzle for all loads");
    const int range = (int)(2 * ((rows - 1) * p.ldx + kChunk));
    const char *corner = p.X + 2L * m0 * p.ldx;
    const unsigned lds0 = (unsigned)reinterpret_cast<uintptr_t>((lds_addr_t)lds);
    auto load_x = [&](int c, int st) {
        const bool inside = c * kChunk + c8 < p.K;
#pragma unroll
        for (int i = 0; i < L; ++i)
            dma16_lowp(corner + 2L * c * kChunk, range, lds0 + st * STAGE + (i * NWAVES + wave) * 1024,
                       (int)(inside && row0 + 4 * NWAVES * i < rows ? off0 + i * step : kOutOfRange));
    };
    // Race-check build (SGEMM_LDS_POISON, see sgemm_lean.hpp): NaN bits into
    // what this lane's loads of stage `st` fill, landed before they are issued.
    auto poison = [&](int st) {
        if constexpr (SGEMM_LDS_POISON) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                *reinterpret_cast<i32x4 *>(lds + st * STAGE + (i * NWAVES + wave) * 1024 + 16 * lane) = i32x4{-1, -1, -1, -1};
            wait_lgkmcnt0();
        }
    };
    // lane (lr, lg) loads for its row of W; the scale of the four columns that
    // a lane's results stand in comes from the lanes that hold them
    const unsigned char *wtile = p.packed + (long)n0 * p.chunks * 64, *ztile = ZEROS ? p.zeros + (long)n0 * p.chunks * GPC : nullptr;
    const unsigned short *stile = p.scales + (long)n0 * p.chunks * GPC;
    unsigned first[NB];                                     // first chunk of the lane's rows, from n0 on
#pragma unroll
    for (int b = 0; b < NB; ++b) first[b] = (unsigned)(min(16 * (wn * NB + b) + lr, p.N - 1 - n0) * p.chunks);
    using Scales = typename std::conditional<GPC == 4, unsigned long, unsigned>::type;
    i32x4 w[NB];
    Scales sc[NB];
    unsigned zp[NB];
    auto load_w = [&](int c) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const unsigned at = first[b] + c;
            w[b] = *reinterpret_cast<const i32x4 *>(wtile + (at * 64 + 16 * lg));
            if constexpr (GPC > 1) sc[b] = *reinterpret_cast<const Scales *>(stile + at * GPC);
            else sc[b] = stile[at];
            if constexpr (ZEROS && GPC == 4) zp[b] = *reinterpret_cast<const unsigned *>(ztile + at * GPC);
            else if constexpr (ZEROS && GPC == 2) zp[b] = *reinterpret_cast<const unsigned short *>(ztile + at * GPC);
            else zp[b] = ZEROS ? ztile[at] : 0x08080808u;
        }
    };
    f32x4 total[MI][NB];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int b = 0; b < NB; ++b) total[mi][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    // the values and scales of k steps h*SPG .. of a chunk, from its registers
    i32x4 wf[2][SPG][NB];
    f32x4 scale[2][NB];
    // word (b, s) of part h, and the scales of part h for block b
    auto unpack_word = [&](auto hc, auto bc, auto sc_, const i32x4 (&cw)[NB], const unsigned (&cz)[NB]) {
        constexpr int h = decltype(hc)::value, b = decltype(bc)::value, s = decltype(sc_)::value;
        const unsigned z = cz[b] >> (8 * (h * GPC / PARTS)) & 255;
        wf[h & 1][s][b] = centred<F16>(cw[b][h * SPG + s], F16 ? (0x4C00u + (z << 6)) * 0x10001u : __float_as_uint((float)z));
    };
    auto unpack_scale = [&](auto hc, auto bc, const Scales (&cs)[NB]) {
        constexpr int h = decltype(hc)::value, b = decltype(bc)::value;
        const float mine = widen16<F16>((unsigned short)(cs[b] >> (16 * (h * GPC / PARTS))));
#pragma unroll
        for (int r = 0; r < 4; ++r) scale[h & 1][b][r] = __shfl(mine, 4 * lg + r);
    };
    const int frag = (wm * MI * 16 + lr) * 256;             // this lane's row in a stage
    auto read_x = [&](const char *stage, int mi, int step) {
        return *reinterpret_cast<const i32x4 *>(stage + frag + mi * 16 * 256 + 16 * ((4 * step + lg) ^ lr));
    };
    if (p.chunks > 0) {
        poison(0);
        load_x(0, 0);
        load_w(0);
        static_for<0, NB>([&](auto bc) {
            unpack_scale(IntC<0>{}, bc, sc);
            static_for<0, SPG>([&](auto s) { unpack_word(IntC<0>{}, bc, s, w, zp); });
        });
    }
    for (int c = 0; c < p.chunks; ++c) {
        // this wave's loads of chunk c have landed, then everyone's; and
        // everyone has read the other stage
        wait_vm_lgkm0<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        i32x4 cw[NB];
        Scales cs[NB];
        unsigned cz[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            cw[b] = w[b];
            cs[b] = used_scales<GROUP>(sc[b], c == p.chunks - 1, p.K);     // (a chunk's first group is taken from sc: it holds a k)
            cz[b] = zp[b];
        }
        const int next = min(c + 1, p.chunks - 1);          // (the last chunk's weights once more, unused)
        poison((c + 1) & 1);
        if (c + 1 < p.chunks) load_x(c + 1, (c + 1) & 1);
        load_w(next);
        __builtin_amdgcn_sched_barrier(0);
        const char *stage = lds + (c & 1) * STAGE;
        // Step j = (part h, 16 rows mi): its matrix instructions; in between,
        // the sums of the step before are scaled, X for step j + AHEAD is
        // read and, spread over the part, the values of the next part (or
        // of the next chunk's first) are unpacked.
        constexpr int STEPS = PARTS * MI, AHEAD = 3;
        f32x4 sum[2][NB];
        i32x4 x[AHEAD + 1][SPG];
        auto read_step = [&](auto jc) {
            constexpr int j = decltype(jc)::value;
#pragma unroll
            for (int s = 0; s < SPG; ++s) x[j % (AHEAD + 1)][s] = read_x(stage, j % MI, j / MI * SPG + s);
        };
        // results of a step, in as many pieces as it has matrix instructions
        constexpr int Q = SPG * NB;
        auto finish = [&](auto jc, auto qc) {
            constexpr int j = decltype(jc)::value, q = decltype(qc)::value;
#pragma unroll
            for (int e = 4 * NB * q / Q; e < 4 * NB * (q + 1) / Q; ++e)
                total[j % MI][e / 4][e % 4] += sum[j & 1][e / 4][e % 4] * scale[j / MI & 1][e / 4][e % 4];
        };
        static_for<0, AHEAD>(read_step);
        __builtin_amdgcn_sched_barrier(0);
        static_for<0, STEPS>([&](auto jc) {
            constexpr int j = decltype(jc)::value, h = j / MI, mi = j % MI, next_h = (h + 1) % PARTS;
            static_for<0, Q>([&](auto qc) {
                constexpr int q = decltype(qc)::value, s = q / NB, b = q % NB;
                sum[j & 1][b] = mfma_16x16x32<F16>(wf[h & 1][s][b], x[j % (AHEAD + 1)][s],
                                                   s == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[j & 1][b]);
                if constexpr (q == 0 && j + AHEAD < STEPS) read_step(IntC<j + AHEAD>{});
                if constexpr (j > 0) finish(IntC<(j > 0 ? j - 1 : 0)>{}, qc);
                // Q words of the next part over the steps mi of this one
                static_for<Q * (mi * Q + q) / (MI * Q), Q * (mi * Q + q + 1) / (MI * Q)>([&](auto uc) {
                    constexpr int u = decltype(uc)::value;
                    if constexpr (u / SPG * SPG == u) unpack_scale(IntC<next_h>{}, IntC<u / SPG>{}, next_h ? cs : sc);
                    unpack_word(IntC<next_h>{}, IntC<u / SPG>{}, IntC<u % SPG>{}, next_h ? cw : w, next_h ? cz : zp);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        static_for<0, Q>([&](auto qc) { finish(IntC<STEPS - 1>{}, qc); });
    }
    constexpr int E = OUT16 ? 2 : 4;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
        const int row = m0 + (wm * MI + mi) * 16 + lr;
        if (row >= p.M) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            store4<F16, OUT16>(p.C + (long)row * p.ldc * E, n0 + (wn * NB + b) * 16 + 4 * lg, p.N, p.beta,
                               total[mi][b] * p.alpha);
    }
}

template <bool F16>
__device__ __forceinline__ unsigned short to16(float v) {
    const f32x4 v4 = {v, v, v, v};
    return (unsigned short)round16<F16>(v4)[0];
}

struct PackArgs {
    const unsigned short *W;            // quantize: in; dequantize: out
    unsigned short *out;
    unsigned char *packed, *zeros;
    unsigned short *scales;
    long ldw;
    int N, K, chunks;
    bool vec;                           // rows of W are whole aligned 16-byte chunks
};

// Eight elements k .. k+7 of a row, zero behind K, two to a register.
__device__ __forceinline__ i32x4 load8(const unsigned short *row, int k, int K, bool vec) {
    i32x4 v = {0, 0, 0, 0};
    if (vec) {
        if (k < K) v = *reinterpret_cast<const i32x4 *>(row + k);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K) v[e >> 1] |= (int)row[k + e] << (16 * (e & 1));
    }
    return v;
}

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// One thread per 32 consecutive k (word (j, s) of a chunk holds k = 32 s + 8 j:
// a thread's four words have its s); the GROUP / 32 threads of a group find its
// extremes together.  s is rounded to 16 bits first and q chosen for the
// rounded s: symmetric s = max|w| / 7, z = 8; with zero points
// s = (max(w, 0) - min(w, 0)) / 15, z = round(-min(w, 0) / s);
// q = round(w / s) + z within 0 .. 15, halves to even.  s == 0 (a group of
// zeros, or one whose s rounds to 0) gives q = z.  A NaN or an infinity in a
// group makes its s NaN.  What does not depend on an element (the place, the
// extremes, s) is done once per 32 of them: 14336 x 4096 42 us, 2.8 TB/s of W;
// a thread per 8 was bound by its vector instructions, at 50.
template <int GROUP, bool ZEROS, bool F16>
__global__ void __launch_bounds__(256) w4_quantize_kernel(PackArgs p) {
    constexpr int TG = GROUP / 32;
    const long per_row = (long)p.chunks * 4, all = per_row * p.N;
    for (long t0 = blockIdx.x * 256L; t0 < all; t0 += gridDim.x * 256L) {       // whole groups: 256 and all are multiples of 4
        const long t = t0 + threadIdx.x;
        if (t >= all) continue;
        const long row = t / per_row;
        const int i = (int)(t - row * per_row);
        i32x4 raw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = load8(p.W + row * p.ldw, 32 * i + 8 * j, p.K, p.vec);
        // The extremes from the bits, two values to an instruction: the largest
        // signed 16-bit integer is the largest value, if any is above 0, the
        // largest unsigned one the most negative, if any is below; then both
        // magnitudes of the group's threads together.
        s16x2 high = {0, 0};
        u16x2 low = {0, 0};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int two = raw[e / 4][e % 4];
            high = __builtin_elementwise_max(high, __builtin_bit_cast(s16x2, two));
            low = __builtin_elementwise_max(low, __builtin_bit_cast(u16x2, two));
        }
        const unsigned top = max((int)high[0], (int)high[1]), bottom = max((unsigned)low[0], (unsigned)low[1]);
        u16x2 both = {(unsigned short)top, (unsigned short)(bottom > 0x8000u ? bottom & 0x7FFFu : 0u)};
#pragma unroll
        for (int d = 1; d < TG; d <<= 1) {
            const int other = __shfl_xor(__builtin_bit_cast(int, both), d);
            both = __builtin_elementwise_max(both, __builtin_bit_cast(u16x2, other));
        }
        const float hi = widen16<F16>(both[0]), lo = widen16<F16>(both[1]);       // lo: -min(w, 0)
        constexpr unsigned short kInfinite = F16 ? 0x7C00 : 0x7F80;
        float s = ZEROS ? (hi + lo) / 15.f : fmaxf(hi, lo) / 7.f;
        if (both[0] >= kInfinite || both[1] >= kInfinite) s = __builtin_nanf("");
        const unsigned short s16 = to16<F16>(s);
        s = widen16<F16>(s16);
        const bool none = !(s > 0.f);                       // 0 or NaN
        const float step = none ? 1.f : s;
        const float z = ZEROS ? (s == s ? fminf(rintf(lo / step), 15.f) : 0.f) : 8.f;
        // round(w / s) without divisions where w * (1 / s), off by less than
        // 2^-17 for |w / s| below 32, lies further than that from a half
        const float inverse = none ? 0.f : __builtin_amdgcn_rcpf(step);
        const int c = i >> 2, run = i & 3;
        unsigned *words = reinterpret_cast<unsigned *>(p.packed + (row * p.chunks + c) * 64 + 4 * run);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            auto value = [&](int e) {
                return widen16<F16>((unsigned short)((unsigned)raw[j][e >> 1] >> (16 * (e & 1))));
            };
            float n[8], far = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = value(e) * inverse;
                n[e] = rintf(x);
                far = fmaxf(far, fabsf(x - n[e]));
            }
            if (!none && (!(far < 0.4999f) || step < 0x1p-100f)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) n[e] = rintf(value(e) / step);
            }
            unsigned word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q = none ? z : fminf(fmaxf(n[e] + z, 0.f), 15.f);
                word |= (unsigned)q << (4 * (e >> 1) + 16 * (e & 1));
            }
            words[4 * j] = word;
        }
        if (i % TG == 0) {
            const long g = row * p.chunks * (kChunk / GROUP) + i / TG;
            p.scales[g] = s16;
            if (ZEROS) p.zeros[g] = (unsigned char)z;
        }
    }
}

template <int GROUP, bool ZEROS, bool F16>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(PackArgs p) {
    constexpr int TG = GROUP / 8;
    const long per_row = (long)p.chunks * 16, all = per_row * p.N;
    for (long t = blockIdx.x * 256L + threadIdx.x; t < all; t += gridDim.x * 256L) {
        const long row = t / per_row;
        const int i = (int)(t - row * per_row), k = 8 * i;
        if (k >= p.K) continue;
        const int c = i >> 4, in = i & 15;
        const unsigned word =
            *reinterpret_cast<const unsigned *>(p.packed + (row * p.chunks + c) * 64 + 16 * (in & 3) + 4 * (in >> 2));
        const long g = row * p.chunks * (kChunk / GROUP) + i / TG;
        const float s = widen16<F16>(p.scales[g]), z = ZEROS ? (float)p.zeros[g] : 8.f;
        i32x4 o;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int e = 4 * h + r;
                v[r] = ((float)(word >> (4 * (e >> 1) + 16 * (e & 1)) & 15) - z) * s;
            }
            const i32x2 x = round16<F16>(v);
            o[2 * h] = x[0];
            o[2 * h + 1] = x[1];
        }
        unsigned short *dst = p.out + row * p.ldw + k;
        if (p.vec) {
            *reinterpret_cast<i32x4 *>(dst) = o;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < p.K) dst[e] = (unsigned short)((unsigned)o[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// f(compile-time group, zeros, fp16)
template <class F>
hipError_t with_form(int group, bool zeros, bool f16, F &&f) {
    auto by_type = [&](auto g, auto z) { return f16 ? f(g, z, std::true_type{}) : f(g, z, std::false_type{}); };
    auto by_zero = [&](auto g) { return zeros ? by_type(g, std::true_type{}) : by_type(g, std::false_type{}); };
    return group == 32 ? by_zero(IntC<32>{}) : group == 64 ? by_zero(IntC<64>{}) : by_zero(IntC<128>{});
}

template <int MB, int NB, int NW>
hipError_t launch_rows(const W4Args &p, int group, bool f16, bool out16, hipStream_t s) {
    const dim3 grid((unsigned)((p.N + 16 * NB - 1) / (16 * NB)), (unsigned)((p.M + 16 * MB - 1) / (16 * MB))), block(64 * NW);
    return with_form(group, p.zeros != nullptr, f16, [&](auto g, auto z, auto f) {
        constexpr int G = decltype(g)::value;
        constexpr bool Z = decltype(z)::value, F = decltype(f)::value;
        return out16 ? launch_k(w4_rows_kernel<MB, NB, NW, G, Z, F, true>, grid, block, s, p)
                     : launch_k(w4_rows_kernel<MB, NB, NW, G, Z, F, false>, grid, block, s, p);
    });
}

template <int MI, int NB, int WM, int WN>
hipError_t launch_tile(const W4Args &p, int group, bool f16, bool out16, hipStream_t s) {
    constexpr int BM = 16 * MI * WM, BN = 16 * NB * WN;
    const dim3 grid((unsigned)(((p.M + BM - 1L) / BM) * ((p.N + BN - 1) / BN))), block(64 * WM * WN);
    return with_form(group, p.zeros != nullptr, f16, [&](auto g, auto z, auto f) {
        constexpr int G = decltype(g)::value;
        constexpr bool Z = decltype(z)::value, F = decltype(f)::value;
        return out16 ? launch_k(w4_tile_kernel<MI, NB, WM, WN, G, Z, F, true>, grid, block, s, p)
                     : launch_k(w4_tile_kernel<MI, NB, WM, WN, G, Z, F, false>, grid, block, s, p);
    });
}

// Up to 64 rows: the widest block of W that still leaves 200 workgroups (more
// columns share the loads of X, fewer workgroups leave compute units idle:
// 8 x 14336 x 4096 18.6 / 16.7 / 14.2 us on 16, 32 and 64 columns, 16 x 8192 x
// 4096 12.7 / 9.3 / 11.8, 1 x 4096 x 4096 5.3 / 6.6 / 10.1).  More rows: the
// shortest of three predicted times, all for K = 4096, per 256 workgroups of a
// kernel once a compute unit's share is full: 32 x 64 blocks of the first
// kernel 19.6 us, 64 x 128 tiles 27 us (41 at least), 128 x 128 tiles 41 us (51
// at least); measured on N = 8192 for 128 rows 37.7 / 42.3 / 51.6 us, for 256
// rows 73.9 / 43.9 / 51.7, for 512 rows - / 59.0 / 53.3, for 2048 rows
// - / 220 / 165 (groups of 64 with zero points; groups of 128 take 36 us for 128
// rows, groups of 32 with zero points 45).
// The forms as sgemm_w4_select_form() numbers them.
enum Form { kRows16x16, kRows16x32, kRows16x64, kRows32x16, kRows32x32, kRows32x64, kTile64x128, kTile128x128 };

Form select_form(int M, int N) {
    auto blocks = [&](int bm, int bn) { return (M + bm - 1L) / bm * ((N + bn - 1L) / bn); };
    if (M <= 16) return blocks(16, 64) >= 200 ? kRows16x64 : blocks(16, 32) >= 200 ? kRows16x32 : kRows16x16;
    const double rows = std::max(19.6, 19.6 * blocks(32, 64) / 256), t64 = std::max(41.0, 27.0 * blocks(64, 128) / 256),
                 t128 = std::max(51.0, 41.0 * blocks(128, 128) / 256);
    if (M <= 64 || (rows <= t64 && rows <= t128))
        return blocks(32, 64) >= 200 ? kRows32x64 : blocks(32, 32) >= 200 ? kRows32x32 : kRows32x16;
    return t64 <= t128 ? kTile64x128 : kTile128x128;
}

// Whether one launch can cover the outputs (the kernel for few rows, which has
// tile rows in gridDim.y, is taken for up to 536 tiles or up to 64 rows).
bool form_fits(int M, int N) {
    switch (select_form(M, N)) {
        case kTile64x128: return launch_fits((M + 63L) / 64 * ((N + 127L) / 128), 256);
        case kTile128x128: return launch_fits((M + 127L) / 128 * ((N + 127L) / 128), 256);
        default: return launch_fits((N + 63L) / 64, 512);
    }
}

hipError_t launch_w4(const W4Args &p, int group, bool f16, bool out16, hipStream_t s) {
    switch (select_form(p.M, p.N)) {
        case kRows16x16: return launch_rows<1, 1, 8>(p, group, f16, out16, s);
        case kRows16x32: return launch_rows<1, 2, 8>(p, group, f16, out16, s);
        case kRows16x64: return launch_rows<1, 4, 8>(p, group, f16, out16, s);
        case kRows32x16: return launch_rows<2, 1, 8>(p, group, f16, out16, s);
        case kRows32x32: return launch_rows<2, 2, 8>(p, group, f16, out16, s);
        case kRows32x64: return launch_rows<2, 4, 4>(p, group, f16, out16, s);
        case kTile64x128: return launch_tile<4, 2, 1, 4>(p, group, f16, out16, s);
        default: return launch_tile<8, 2, 1, 4>(p, group, f16, out16, s);
    }
}

int check(int dtype, int N, int K, int group) {
    if (dtype != SGEMM_DTYPE_BF16 && dtype != SGEMM_DTYPE_F16) return SGEMM_STATUS_INVALID_DTYPE;
    if (N < 0 || K < 0 || (group != 32 && group != 64 && group != 128)) return SGEMM_STATUS_INVALID_DIM;
    return K > kMaxLd16 || N > (1 << 30) ? SGEMM_STATUS_INVALID_DIM : SGEMM_STATUS_OK;
}

constexpr int kMaxRows = 1 << 24;       // launch grid extents

// The packed form's alignment: a chunk of weights, scales and zero points each in one load.
bool packed_ok(const void *packed, const void *scales, const void *zeros) {
    return !(reinterpret_cast<uintptr_t>(packed) & 15) && !(reinterpret_cast<uintptr_t>(scales) & 7) &&
           !(reinterpret_cast<uintptr_t>(zeros) & 3);
}

int chunks_of(int K) { return (K + kChunk - 1) / kChunk; }

unsigned pack_blocks(long threads) { return (unsigned)std::min((threads + 255) / 256, 8192L); }

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

long long sgemm_w4_workspace(int M, int K, const void *X, int ldx) {
    if (M < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    return M == 0 || K == 0 || chunk_rows(X, ldx, K) ? 0 : 2L * M * ceil_to(K, 8);
}

int sgemm_w4(int dtype, int M, int N, int K, float alpha, const void *X, int ldx, const void *packed,
             const void *scales, const void *zeros, int group, float beta, void *C, int ldc, int dtype_c,
             void *workspace, long long workspace_bytes, void *stream) {
    const int st = check(dtype, N, K, group);
    if (st != SGEMM_STATUS_OK) return st;
    if (dtype_c != dtype && dtype_c != SGEMM_DTYPE_F32) return SGEMM_STATUS_INVALID_DTYPE;
    if (M < 0 || M > kMaxRows || ldx < std::max(K, 1) || ldc < std::max(N, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (!form_fits(M, N)) return SGEMM_STATUS_INVALID_DIM;
    if (M == 0 || N == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || (K > 0 && (X == nullptr || packed == nullptr || scales == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    if (!packed_ok(packed, scales, zeros)) return SGEMM_STATUS_UNSUPPORTED;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    W4Args p = {static_cast<const char *>(X), static_cast<const unsigned char *>(packed),
                static_cast<const unsigned char *>(zeros), static_cast<const unsigned short *>(scales),
                static_cast<char *>(C), ldx, ldc, M, N, K, chunks_of(K), alpha, beta};
    const bool f16 = dtype == SGEMM_DTYPE_F16, out16 = dtype_c != SGEMM_DTYPE_F32;
    const long long copy = sgemm_w4_workspace(M, K, X, ldx);
    if (copy > 0) {
        if (workspace == nullptr || workspace_bytes < copy || (reinterpret_cast<uintptr_t>(workspace) & 15))
            return SGEMM_STATUS_SCRATCH_TOO_SMALL;
        const hipError_t e = pad_rows(X, ldx, 0, 1, M, K, workspace, s);
        if (e != hipSuccess) return hip_status(e, "kernel launch");
        p.X = static_cast<const char *>(workspace);
        p.ldx = ceil_to(K, 8);
        p.K = (int)p.ldx;                   // the copy's columns behind K are zeros
    }
    const hipError_t e = launch_w4(p, group, f16, out16, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_w4_select_form(int M, int N) {
    return M < 0 || N < 0 ? SGEMM_STATUS_INVALID_DIM : select_form(M, N);
}

int sgemm_w4_quantize(int dtype, int N, int K, const void *W, int ldw, int group, void *packed, void *scales,
                      void *zeros, void *stream) {
    const int st = check(dtype, N, K, group);
    if (st != SGEMM_STATUS_OK) return st;
    if (ldw < std::max(K, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (N == 0 || K == 0) return SGEMM_STATUS_OK;
    if (W == nullptr || packed == nullptr || scales == nullptr) return SGEMM_STATUS_NULL_POINTER;
    if (!packed_ok(packed, scales, zeros)) return SGEMM_STATUS_UNSUPPORTED;
    const PackArgs p = {static_cast<const unsigned short *>(W), nullptr, static_cast<unsigned char *>(packed),
                        static_cast<unsigned char *>(zeros), static_cast<unsigned short *>(scales), ldw, N, K,
                        chunks_of(K), (reinterpret_cast<uintptr_t>(W) & 15) == 0 && ldw % 8 == 0 && K % 8 == 0};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = with_form(group, zeros != nullptr, dtype == SGEMM_DTYPE_F16, [&](auto g, auto z, auto f) {
        return launch_k(w4_quantize_kernel<decltype(g)::value, decltype(z)::value, decltype(f)::value>,
                        dim3(pack_blocks(p.N * p.chunks * 4L)), dim3(256), s, p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_w4_dequantize(int dtype, int N, int K, const void *packed, const void *scales, const void *zeros, int group,
                        void *W, int ldw, void *stream) {
    const int st = check(dtype, N, K, group);
    if (st != SGEMM_STATUS_OK) return st;
    if (ldw < std::max(K, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (N == 0 || K == 0) return SGEMM_STATUS_OK;
    if (W == nullptr || packed == nullptr || scales == nullptr) return SGEMM_STATUS_NULL_POINTER;
    if (!packed_ok(packed, scales, zeros)) return SGEMM_STATUS_UNSUPPORTED;
    const PackArgs p = {nullptr, static_cast<unsigned short *>(W),
                        const_cast<unsigned char *>(static_cast<const unsigned char *>(packed)),
                        const_cast<unsigned char *>(static_cast<const unsigned char *>(zeros)),
                        const_cast<unsigned short *>(static_cast<const unsigned short *>(scales)), ldw, N, K,
                        chunks_of(K), (reinterpret_cast<uintptr_t>(W) & 15) == 0 && ldw % 8 == 0 && K % 8 == 0};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = with_form(group, zeros != nullptr, dtype == SGEMM_DTYPE_F16, [&](auto g, auto z, auto f) {
        return launch_k(w4_dequantize_kernel<decltype(g)::value, decltype(z)::value, decltype(f)::value>,
                        dim3(pack_blocks(p.N * p.chunks * 16L)), dim3(256), s, p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

}  // extern "C"

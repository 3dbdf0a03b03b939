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
// multiply-add per output and group.
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

// The two 16-bit values 16 + q of nibble i of each half of a word.
template <bool F16, int I>
__device__ __forceinline__ int q_pair(unsigned w) {
    constexpr int to = (F16 ? 6 : 3) - 4 * I;              // shift left
    const unsigned v = to >= 0 ? w << (to >= 0 ? to : 0) : w >> (to < 0 ? -to : 0);
    return (int)((v & (F16 ? 0x03C003C0u : 0x00780078u)) | (F16 ? 0x4C004C00u : 0x41804180u));
}

// MB blocks of 16 rows of X by 16 rows of W per workgroup; its NW waves
// share the chunks and add up through LDS.  GROUP: k per scale.  XVEC: rows
// of X are whole aligned 16-byte chunks.
template <int MB, int NW, int GROUP, bool ZEROS, bool F16, bool OUT16, bool XVEC>
__global__ void __launch_bounds__(64 * NW) w4_kernel(W4Args p) {
    constexpr int GPC = kChunk / GROUP, SPG = 4 / GPC;      // groups per chunk, k steps per group
    __shared__ f32x4 part[NW][MB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MB;
    const long n = min(n0 + lr, p.N - 1);
    const unsigned char *wrow = p.packed + n * p.chunks * 64 + 16 * lg;
    const unsigned short *srow = p.scales + n * p.chunks * GPC;
    const unsigned char *zrow = ZEROS ? p.zeros + n * p.chunks * GPC : nullptr;
    const unsigned short *xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
        xrow[b] = reinterpret_cast<const unsigned short *>(p.X) + (long)min(m0 + 16 * b + lr, p.M - 1) * p.ldx;
    const int one = F16 ? 0x3C003C00 : 0x3F803F80;
    const i32x4 ones = {one, one, one, one};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 total[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) total[b] = zero;
    for (int c = wave; c < p.chunks; c += NW) {
        const i32x4 w = *reinterpret_cast<const i32x4 *>(wrow + (long)c * 64);
        f32x4 sum[MB], sx[MB];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = c * kChunk + 32 * s + 8 * lg;
            const i32x4 wf = {q_pair<F16, 0>(w[s]), q_pair<F16, 1>(w[s]), q_pair<F16, 2>(w[s]), q_pair<F16, 3>(w[s])};
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                i32x4 xf = {0, 0, 0, 0};
                if constexpr (XVEC) {
                    if (k < p.K) xf = *reinterpret_cast<const i32x4 *>(xrow[b] + k);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (k + e < p.K) xf[e >> 1] |= (int)xrow[b][k + e] << (16 * (e & 1));
                }
                sum[b] = mfma_16x16x32<F16>(xf, wf, s % SPG == 0 ? zero : sum[b]);
                sx[b] = mfma_16x16x32<F16>(xf, ones, s % SPG == 0 ? zero : sx[b]);
            }
            if (s % SPG == SPG - 1) {
                const int g = c * GPC + s / SPG;
                const float scale = widen16<F16>(srow[g]), z = ZEROS ? 16.f + (float)zrow[g] : 24.f;
#pragma unroll
                for (int b = 0; b < MB; ++b) total[b] += (sum[b] - sx[b] * z) * scale;
            }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) part[wave][b][lane] = total[b];
    __syncthreads();
    // block b's lane l holds rows 4*(l/16) .. +3 of column l%16
    for (int t = threadIdx.x; t < MB * 64; t += 64 * NW) {
        const int b = t >> 6, l = t & 63;
        f32x4 v = part[0][b][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w][b][l];
        const int col = n0 + (l & 15);
        if (col >= p.N) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = m0 + 16 * b + 4 * (l >> 4) + r;
            if (row >= p.M) continue;
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

// Eight elements k .. k+7 of a row, zero behind K.
__device__ __forceinline__ void load8(const unsigned short *row, int k, int K, bool vec, unsigned short (&v)[8]) {
    typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
    if (vec && k < K) {
        const u16x8 x = *reinterpret_cast<const u16x8 *>(row + k);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < K ? row[k + e] : (unsigned short)0;
    }
}

// One thread per 8 consecutive k; the GROUP / 8 threads of a group find its
// extremes together.  s is rounded to 16 bits first and q chosen for the
// rounded s: symmetric s = max|w| / 7, z = 8; with zero points
// s = (max(w, 0) - min(w, 0)) / 15, z = round(-min(w, 0) / s);
// q = round(w / s) + z within 0 .. 15, halves to even.  s == 0 (a group of
// zeros, or one whose s rounds to 0) gives q = z.  A NaN or an infinity in a
// group makes its s NaN.
template <int GROUP, bool ZEROS, bool F16>
__global__ void __launch_bounds__(256) w4_quantize_kernel(PackArgs p) {
    constexpr int TG = GROUP / 8;
    const long per_row = (long)p.chunks * 16, all = per_row * p.N;
    for (long t0 = blockIdx.x * 256L; t0 < all; t0 += gridDim.x * 256L) {       // whole groups: 256 and all are multiples of 16
        const long t = t0 + threadIdx.x;
        if (t >= all) continue;
        const long row = t / per_row;
        const int i = (int)(t - row * per_row), k = 8 * i;
        unsigned short raw[8];
        load8(p.W + row * p.ldw, k, p.K, p.vec, raw);
        float w[8], lo = 0.f, hi = 0.f;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = widen16<F16>(raw[e]);
            lo = fminf(lo, w[e]);
            hi = fmaxf(hi, w[e]);
            bad |= !(fabsf(w[e]) < __builtin_inff());
        }
        if (bad) hi = __builtin_inff();
#pragma unroll
        for (int d = 1; d < TG; d <<= 1) {
            lo = fminf(lo, __shfl_xor(lo, d));
            hi = fmaxf(hi, __shfl_xor(hi, d));
        }
        float s = ZEROS ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
        if (hi == __builtin_inff()) s = __builtin_nanf("");
        const unsigned short s16 = to16<F16>(s);
        s = widen16<F16>(s16);
        const bool none = !(s > 0.f);                       // 0 or NaN
        const float step = none ? 1.f : s;
        const float z = ZEROS ? (s == s ? fminf(rintf(-lo / step), 15.f) : 0.f) : 8.f;
        unsigned word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = none ? z : fminf(fmaxf(rintf(w[e] / step) + z, 0.f), 15.f);
            word |= (unsigned)q << (4 * (e >> 1) + 16 * (e & 1));
        }
        const int c = i >> 4, in = i & 15;                  // word s = in / 4 of run j = in % 4
        *reinterpret_cast<unsigned *>(p.packed + (row * p.chunks + c) * 64 + 16 * (in & 3) + 4 * (in >> 2)) = word;
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

template <int MB, int NW>
hipError_t launch_w4(const W4Args &p, int group, bool f16, bool out16, bool xvec, hipStream_t s) {
    const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 16 * MB - 1) / (16 * MB))), block(64 * NW);
    return with_form(group, p.zeros != nullptr, f16, [&](auto g, auto z, auto f) {
        constexpr int G = decltype(g)::value;
        constexpr bool Z = decltype(z)::value, F = decltype(f)::value;
        if (out16) return xvec ? launch_k(w4_kernel<MB, NW, G, Z, F, true, true>, grid, block, s, p)
                               : launch_k(w4_kernel<MB, NW, G, Z, F, true, false>, grid, block, s, p);
        return xvec ? launch_k(w4_kernel<MB, NW, G, Z, F, false, true>, grid, block, s, p)
                    : launch_k(w4_kernel<MB, NW, G, Z, F, false, false>, grid, block, s, p);
    });
}

int check(int dtype, int N, int K, int group) {
    if (dtype != SGEMM_DTYPE_BF16 && dtype != SGEMM_DTYPE_F16) return SGEMM_STATUS_INVALID_DTYPE;
    if (N < 0 || K < 0 || (group != 32 && group != 64 && group != 128)) return SGEMM_STATUS_INVALID_DIM;
    return K > (1 << 30) ? SGEMM_STATUS_INVALID_DIM : SGEMM_STATUS_OK;
}

int chunks_of(int K) { return (K + kChunk - 1) / kChunk; }

unsigned pack_blocks(const PackArgs &p) { return (unsigned)std::min((p.N * p.chunks * 16L + 255) / 256, 8192L); }

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

int sgemm_w4(int dtype, int M, int N, int K, float alpha, const void *X, int ldx, const void *packed,
             const void *scales, const void *zeros, int group, float beta, void *C, int ldc, int dtype_c,
             void *stream) {
    const int st = check(dtype, N, K, group);
    if (st != SGEMM_STATUS_OK) return st;
    if (dtype_c != dtype && dtype_c != SGEMM_DTYPE_F32) return SGEMM_STATUS_INVALID_DTYPE;
    if (M < 0 || ldx < std::max(K, 1) || ldc < std::max(N, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (M == 0 || N == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || (K > 0 && (X == nullptr || packed == nullptr || scales == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(packed) & 15) return SGEMM_STATUS_UNSUPPORTED;
    if ((M + 15) / 16 > 65535) return SGEMM_STATUS_INVALID_DIM;
    const W4Args p = {static_cast<const char *>(X), static_cast<const unsigned char *>(packed),
                      static_cast<const unsigned char *>(zeros), static_cast<const unsigned short *>(scales),
                      static_cast<char *>(C), ldx, ldc, M, N, K, chunks_of(K), alpha, beta};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool f16 = dtype == SGEMM_DTYPE_F16, out16 = dtype_c != SGEMM_DTYPE_F32;
    const bool xvec = (reinterpret_cast<uintptr_t>(X) & 15) == 0 && ldx % 8 == 0 && K % 8 == 0;
    const hipError_t e = M <= 16 ? launch_w4<1, 8>(p, group, f16, out16, xvec, s)
                                 : launch_w4<4, 4>(p, group, f16, out16, xvec, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_w4_quantize(int dtype, int N, int K, const void *W, int ldw, int group, void *packed, void *scales,
                      void *zeros, void *stream) {
    const int st = check(dtype, N, K, group);
    if (st != SGEMM_STATUS_OK) return st;
    if (ldw < std::max(K, 1)) return SGEMM_STATUS_INVALID_DIM;
    if (N == 0 || K == 0) return SGEMM_STATUS_OK;
    if (W == nullptr || packed == nullptr || scales == nullptr) return SGEMM_STATUS_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(packed) & 15) return SGEMM_STATUS_UNSUPPORTED;
    const PackArgs p = {static_cast<const unsigned short *>(W), nullptr, static_cast<unsigned char *>(packed),
                        static_cast<unsigned char *>(zeros), static_cast<unsigned short *>(scales), ldw, N, K,
                        chunks_of(K), (reinterpret_cast<uintptr_t>(W) & 15) == 0 && ldw % 8 == 0 && K % 8 == 0};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = with_form(group, zeros != nullptr, dtype == SGEMM_DTYPE_F16, [&](auto g, auto z, auto f) {
        return launch_k(w4_quantize_kernel<decltype(g)::value, decltype(z)::value, decltype(f)::value>,
                        dim3(pack_blocks(p)), dim3(256), s, p);
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
    if (reinterpret_cast<uintptr_t>(packed) & 15) return SGEMM_STATUS_UNSUPPORTED;
    const PackArgs p = {nullptr, static_cast<unsigned short *>(W),
                        const_cast<unsigned char *>(static_cast<const unsigned char *>(packed)),
                        const_cast<unsigned char *>(static_cast<const unsigned char *>(zeros)),
                        const_cast<unsigned short *>(static_cast<const unsigned short *>(scales)), ldw, N, K,
                        chunks_of(K), (reinterpret_cast<uintptr_t>(W) & 15) == 0 && ldw % 8 == 0 && K % 8 == 0};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = with_form(group, zeros != nullptr, dtype == SGEMM_DTYPE_F16, [&](auto g, auto z, auto f) {
        return launch_k(w4_dequantize_kernel<decltype(g)::value, decltype(z)::value, decltype(f)::value>,
                        dim3(pack_blocks(p)), dim3(256), s, p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

}  // extern "C"

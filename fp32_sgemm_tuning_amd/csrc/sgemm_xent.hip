// The output layer of a language model with its softmax cross entropy:
// logits l = alpha * X * W^T for rows X [M,K] and a vocabulary W [N,K] in 16
// bits, lse_i = log(sum_v exp(l_iv)), loss_i = lse_i - l_{i,target_i}, and
// the gradients of sum(dloss_i * loss_i)
//
//   dX = alpha * diag(dloss) * P * W,  dW = alpha * P^T * diag(dloss) * X,
//   P_iv = exp(l_iv - lse_i) - [v == target_i]
//
// without the M x N logits ever being in memory.  Rows whose target is the
// ignored index take no part: xent_compact_kernel lists the others and, if
// there is an ignored row, copies them side by side, so no product is spent
// on them and nothing they hold (NaN, Inf) reaches dW.
//
// Forward: each block tile of the logits stays in the accumulators;
// stats_tile writes per row and 128 columns the maximum and the sum of
// exp(l - maximum), and xent_join_kernel joins a row's.
//
// Backward, for one piece of the vocabulary after the other:
// dlogits_tile forms the piece of the logits again and stores
// P_iv * dloss_i / max|dloss| in 16 bits, then xent_dx_kernel adds its
// product with the piece of W to an FP32 sum, and dw_tile writes the piece of
// dW.  P lies in [-1, 1] and the scaled dloss too, so the top of the 16-bit
// range is never passed whatever the loss is scaled by; the factor max|dloss|
// is put back in FP32.  Rounding this product to the inputs' 16 bits is what
// lets the two gradient products run on the 16-bit matrix instructions; it is
// off by at most half a step of each term (bf16 2^-8, fp16 2^-11 relative to
// the term), the size of the gradients' own final rounding.
//
// FP16 has no values below 2^-24 and only ones with fewer bits below 2^-14,
// where most of P lies.  There P is stored times 2^15, powers of two stand in
// place of max|dloss| (the next above it), and a row whose |dloss| is below 2^-6
// of that is stored over the next power above its own |dloss|, so that its dX
// does not depend on the other rows': a term is off by 2^-11 of itself or, if
// that is more, 2^-34 of its row's |dloss|.  Before the product of dW, which
// sums over the rows, xent_rescale_kernel brings such rows to the common power:
// its terms are off by 2^-11 of themselves or 2^-39 of max|dloss|.
#include <algorithm>

#include "sgemm_tile16.hpp"

namespace sgemm_mi355x {

namespace {

// In the workspace, per call.  `rows`: rows that are not ignored.
struct XentHead {
    int rows;
    float gmax;        // max |dloss| over them, FP16: the power of two above it; 1 where that is 0 or infinite
};

struct XentArgs {
    const char *X, *W;                  // W: padded copy if one is needed
    long ldx, ldw;
    int M, N, K;
    float alpha;
    const long long *target;
    long long ignore;
    XentHead *head;
    int *map;                           // row of X of each listed row
    int *label;                         // its target, -1 outside 0 .. N-1
    int *seg_rows;                      // many rows: listed rows and max |dloss| per kSegment rows
    float *seg_max;
    char *Xc;                           // the listed rows side by side, K rounded up to whole chunks
    long ldxc;
    bool take_x;                        // X can be used in place if no row is ignored
    bool direct;                        // forward: all rows in place, nothing is listed
    float *loss, *lse;
    // forward
    float *tlogit;                      // logit of the target, per listed row
    float2 *part;                       // [128 columns][listed row]: maximum, sum
    // backward
    const float *lse_in, *dloss;
    long dloss_stride;
    bool f16;
    float *g, *lsec;                    // of the listed rows: what P is multiplied by, its lse
    float *back, *down;                 // what their dX is multiplied by, what P for dW
    char *dX, *dW, *P;
    long lddx, lddw, ldp;
    float *sum;                         // FP32 sum of dX over the pieces
    int n_first, n_count;               // piece of the vocabulary
};

__device__ __forceinline__ float max_abs(float a, float b) { return fmaxf(a, fabsf(b)); }

constexpr int kCompactRows = 16, kSegment = 1024;
constexpr int kOnePass = 16384;     // rows up to which a block counts all before it by itself

// Adds up the rows [from, to) that are not ignored, those of them before r0,
// and max|dloss|; eight rows of a thread at a time, so that their loads overlap.
template <bool GRAD>
__device__ __forceinline__ void count_rows(const XentArgs &p, int from, int to, int r0, int &all, int &before, float &gm) {
    for (int i0 = from + threadIdx.x; i0 < to; i0 += 8 * 256) {
        long long t[8];
        float d[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + 256 * u, at = min(i, to - 1);
            t[u] = i < to ? p.target[at] : p.ignore;
            d[u] = GRAD ? p.dloss[at * p.dloss_stride] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (t[u] == p.ignore) continue;
            ++all;
            before += i0 + 256 * u < r0;
            gm = max_abs(gm, d[u]);
        }
    }
}

// Sums of two counts and a maximum over the 256 threads of a block.
__device__ __forceinline__ void block_sums(int &a, int &b, float &m) {
    __shared__ int sa[4], sb[4];
    __shared__ float sm[4];
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        a += __shfl_xor(a, d);
        b += __shfl_xor(b, d);
        m = fmaxf(m, __shfl_xor(m, d));
    }
    if ((threadIdx.x & 63) == 0) {
        sa[threadIdx.x >> 6] = a;
        sb[threadIdx.x >> 6] = b;
        sm[threadIdx.x >> 6] = m;
    }
    __syncthreads();
    a = sa[0] + sa[1] + sa[2] + sa[3];
    b = sb[0] + sb[1] + sb[2] + sb[3];
    m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
}

// Many rows: what xent_compact_kernel needs of each segment.
template <bool GRAD>
__global__ void __launch_bounds__(256) xent_segments_kernel(XentArgs p) {
    int all = 0, before = 0;
    float gm = 0.f;
    const int from = blockIdx.x * kSegment;
    count_rows<GRAD>(p, from, min(from + kSegment, p.M), 0, all, before, gm);
    block_sums(all, before, gm);
    if (threadIdx.x == 0) {
        p.seg_rows[blockIdx.x] = all;
        p.seg_max[blockIdx.x] = gm;
    }
}

// What P is stored times (P and dloss / gmax are at most 1).
constexpr float p_scale(bool f16) { return f16 ? 0x1p15f : 1.f; }

// The power of two above |d|.
__device__ __forceinline__ float power_above(float d) {
    int e;
    (void)frexpf(d, &e);
    return ldexpf(1.f, min(e, 127));
}

// Block b lists the rows b * kCompactRows ...: it counts the rows before
// them itself (a pass over the targets, which stay in L2, so one launch does;
// with many rows over the segments' counts and its own segment).  GRAD: also
// max|dloss|, each listed row's dloss and lse, and zeros in dX for ignored
// rows; else zeros in loss and lse.
template <bool GRAD>
__global__ void __launch_bounds__(256) xent_compact_kernel(XentArgs p) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r0 = blockIdx.x * kCompactRows;
    int nb = 0, na = 0;
    float gm = 0.f;
    if (p.M <= kOnePass) {
        count_rows<GRAD>(p, 0, p.M, r0, na, nb, gm);
    } else {
        const int segment = r0 / kSegment, from = segment * kSegment;
        int own = 0;
        float ignored = 0.f;
        count_rows<GRAD>(p, from, min(from + kSegment, p.M), r0, own, nb, ignored);
        for (int i = tid; i < (p.M + kSegment - 1) / kSegment; i += 256) {
            const int rows = p.seg_rows[i];
            na += rows;
            if (i < segment) nb += rows;
            gm = fmaxf(gm, p.seg_max[i]);
        }
    }
    block_sums(na, nb, gm);
    if (!(gm > 0.f && gm < __builtin_inff())) gm = 1.f;
    else if (GRAD && p.f16) gm = power_above(gm);
    if (blockIdx.x == 0 && tid == 0) *p.head = {na, gm};
    const bool copy = !(p.take_x && na == p.M);
    // each wave: every fourth row
    const int mine = r0 + (lane & (kCompactRows - 1));
    const long long t = mine < p.M ? p.target[mine] : p.ignore;
    const unsigned listed = (unsigned)__ballot(t != p.ignore);        // bit r: row r0 + r
    for (int r = wave; r < kCompactRows && r0 + r < p.M; r += 4) {
        const int row = r0 + r;
        if (!(listed >> r & 1)) {
            if (GRAD) {
                if (p.dX != nullptr)
                    for (int k = 4 * lane; k < p.K; k += 256)
                        store4<false, true>(p.dX + 2 * row * p.lddx, k, p.K, 0.f, f32x4{0.f, 0.f, 0.f, 0.f});
            } else if (lane == 0) {
                p.loss[row] = 0.f;
                p.lse[row] = 0.f;
            }
            continue;
        }
        const int at = nb + __builtin_popcount(listed & ((1u << r) - 1));
        if (lane == 0) {
            const long long v = p.target[row];
            p.map[at] = row;
            p.label[at] = v >= 0 && v < p.N ? (int)v : -1;
            if (GRAD) {
                const float d = p.dloss[row * p.dloss_stride];
                float base = gm;
                if (p.f16) {
                    const float share = fabsf(d / gm);          // (above 1 next to an infinite one)
                    if ((share < 0x1p-6f && d != 0.f) || (share > 1.f && share < __builtin_inff())) base = power_above(d);
                    p.down[at] = base / gm;
                }
                // a target outside the vocabulary: NaN, as its loss is
                p.g[at] = v >= 0 && v < p.N ? d / base * p_scale(p.f16) : __builtin_nanf("");
                p.back[at] = base / p_scale(p.f16);
                p.lsec[at] = p.lse_in[row];
            }
        }
        if (copy) {
            const unsigned short *src = reinterpret_cast<const unsigned short *>(p.X) + row * p.ldx;
            unsigned short *dst = reinterpret_cast<unsigned short *>(p.Xc) + at * p.ldxc;
            for (int k = 8 * lane; k < p.K; k += 512) {             // (rows of any alignment)
                unsigned short v[8];
                if (k + 8 <= p.K) {
                    __builtin_memcpy(v, src + k, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = k + e < p.K ? src[k + e] : (unsigned short)0;
                }
                __builtin_memcpy(__builtin_assume_aligned(dst + k, 16), v, 16);
            }
        }
    }
}

// The listed rows as an operand: X itself if every row is listed.
__device__ __forceinline__ void listed_rows(const XentArgs &p, int rows, const char *&X, long &ldx) {
    const bool in_place = p.take_x && rows == p.M;              // (as `direct` has it)
    X = in_place ? p.X : p.Xc;
    ldx = in_place ? p.ldx : p.ldxc;
}

// The number of listed rows; the target of listed row `row`, -1 outside the
// vocabulary.
__device__ __forceinline__ int listed_count(const XentArgs &p) { return p.direct ? p.M : p.head->rows; }
__device__ __forceinline__ int label_of(const XentArgs &p, int row) {
    if (!p.direct) return p.label[row];
    const long long t = p.target[row];
    return t >= 0 && t < p.N ? (int)t : -1;
}

// The logits (before alpha) of the tile at (m0, n0) of the listed rows by the
// piece of the vocabulary.
template <class T, bool F16>
__device__ __forceinline__ void logits_tile(const XentArgs &p, int rows, char *lds, int m0, int n0,
                                            f32x4 (&acc)[T::MI][T::NB]) {
    Operands16 q = {nullptr, p.W + 2L * p.n_first * p.ldw, 0, p.ldw, rows, p.n_count, p.K};
    listed_rows(p, rows, q.A, q.lda);
    accumulate16<T, F16, false, true>(q, m0, n0, lds, acc);
}

// A row's maximum and sum over each 128 columns of the tile (one slot of
// `part` each, whatever the tile), and the target's logit.
template <class T, bool F16>
__device__ __forceinline__ void stats_tile(const XentArgs &p, int rows, char *lds, int m0, int n0) {
    f32x4 acc[T::MI][T::NB];
    logits_tile<T, F16>(p, rows, lds, m0, n0, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
    const int col0 = n0 + wn * T::WN + 4 * (lane >> 4);
    float2 *red = reinterpret_cast<float2 *>(lds);                  // [WAVES_N][BM]
    __syncthreads();                                                // the K loop's last LDS reads
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
        const int r = wm * T::WM + mi * 16 + (lane & 15), row = m0 + r;
        const int label = row < rows ? label_of(p, row) : -1;
        float top = -__builtin_inff();
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = col0 + nb * 16 + e;
                const float l = acc[mi][nb][e] * p.alpha;
                if (col == label) p.tlogit[row] = l;
                acc[mi][nb][e] = col < p.N ? l : -__builtin_inff();
                top = fmaxf(top, acc[mi][nb][e]);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // (a row of nothing but -inf sums to 0, one with a NaN to NaN)
        const float base = top == -__builtin_inff() ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += __expf(acc[mi][nb][e] - base);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (lane < 16) red[wn * T::BM + r] = make_float2(top, sum);
    }
    __syncthreads();
    constexpr int PER = 128 / T::WN;                                // waves per 128 columns
    for (int t = threadIdx.x; t < T::BM * (T::BN / 128); t += T::NT) {
        const int r = t % T::BM, slot = t / T::BM;
        if (m0 + r >= rows || n0 + 128 * slot >= p.N) continue;
        float2 a = red[slot * PER * T::BM + r];
#pragma unroll
        for (int w = 1; w < PER; ++w) {
            const float2 b = red[(slot * PER + w) * T::BM + r];
            const float top = fmaxf(a.x, b.x), base = top == -__builtin_inff() ? 0.f : top;
            a = make_float2(top, a.y * __expf(a.x - base) + b.y * __expf(b.x - base));
        }
        p.part[(long)(n0 / 128 + slot) * p.M + m0 + r] = a;
    }
}

// Joins the tile columns of 16 rows per block: 64 threads a row take every
// 64th tile, four loads at a time, then a tree.
__global__ void __launch_bounds__(1024) xent_join_kernel(XentArgs p, int tiles_n) {
    __shared__ float2 red[64][16];
    const int r = threadIdx.x & 15, slice = threadIdx.x >> 4, row = blockIdx.x * 16 + r;
    const bool live = row < listed_count(p);
    auto join = [](float2 a, float2 b) {
        const float top = fmaxf(a.x, b.x), base = top == -__builtin_inff() ? 0.f : top;
        return make_float2(top, a.y * __expf(a.x - base) + b.y * __expf(b.x - base));
    };
    const float2 none = make_float2(-__builtin_inff(), 0.f);
    float2 a = none;
    if (live)
        for (int t = slice; t < tiles_n; t += 256) {
            float2 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = t + 64 * i < tiles_n ? p.part[(long)(t + 64 * i) * p.M + row] : none;
            a = join(a, join(join(b[0], b[1]), join(b[2], b[3])));
        }
    red[slice][r] = a;
    for (int half = 32; half; half >>= 1) {
        __syncthreads();
        if (slice < half) red[slice][r] = a = join(a, red[slice + half][r]);
    }
    if (slice != 0 || !live) return;
    const float lse = a.x + logf(a.y);
    const int to = p.direct ? row : p.map[row];
    const bool ignored = p.direct && p.target[row] == p.ignore;
    p.lse[to] = ignored ? 0.f : lse;
    p.loss[to] = ignored ? 0.f : lse - (label_of(p, row) < 0 ? __builtin_nanf("") : p.tlogit[row]);
}

// P [listed rows][piece of the vocabulary] in 16 bits, zeros behind the
// vocabulary's end up to the tile's.
template <class T, bool F16>
__device__ __forceinline__ void dlogits_tile(const XentArgs &p, int rows, char *lds, int m0, int n0) {
    f32x4 acc[T::MI][T::NB];
    logits_tile<T, F16>(p, rows, lds, m0, n0, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col0 = n0 + wave % T::WAVES_N * T::WN + 4 * (lane >> 4);
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
        const int row = m0 + wave / T::WAVES_N * T::WM + mi * 16 + (lane & 15);
        if (row >= rows) continue;
        const int label = p.label[row] - p.n_first;
        const float g = p.g[row], lse = p.lsec[row];
        char *dst = p.P + 2 * row * p.ldp;
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) {
            const int col = col0 + nb * 16;
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float s = __expf(acc[mi][nb][e] * p.alpha - lse) - (col + e == label ? 1.f : 0.f);
                // (dloss 0 takes a row out whatever its logits are)
                v[e] = col + e < p.n_count && g != 0.f ? s * g : 0.f;
            }
            *reinterpret_cast<i32x2 *>(dst + 2 * col) = round16<F16>(v);
        }
    }
}

// The piece of dW: P^T * X over the listed rows.
template <class T, bool F16>
__device__ __forceinline__ void dw_tile(const XentArgs &p, int rows, char *lds, int m0, int n0) {
    Operands16 q = {p.P, nullptr, p.ldp, 0, p.n_count, p.K, rows};
    listed_rows(p, rows, q.B, q.ldb);
    f32x4 acc[T::MI][T::NB];
    accumulate16<T, F16, true, false>(q, m0, n0, lds, acc);
    store_tile<T, F16, true>(acc, m0, n0, p.n_count, p.K, p.dW + 2L * p.n_first * p.lddw, p.lddw,
                             p.alpha * (p.head->gmax / p_scale(F16)), 0.f);
}

// FP16, between the products of dX and of dW: the rows of P that stand for
// dloss over a power of two of their own become shares of gmax like the others.
// As a rule none do (8192 rows by 16128 columns: 5.5 us); where nearly all do
// it is bound by reading and writing P (66 us, beside 800 for the product).
__global__ void __launch_bounds__(256) xent_rescale_kernel(XentArgs p) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const int rows = p.head->rows;
    for (int row = blockIdx.x; row < rows; row += gridDim.x) {
        const float down = p.down[row];
        if (down == 1.f) continue;
        h8 *at = reinterpret_cast<h8 *>(p.P + 2 * row * p.ldp);
        for (int c = blockIdx.y * 256 + threadIdx.x; 8 * c < p.n_count; c += gridDim.y * 256) {
            h8 v = at[c];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (_Float16)((float)v[e] * down);
            at[c] = v;
        }
    }
}

// STEP 0: stats_tile, 1: dlogits_tile, over the listed rows by the piece; 2:
// dw_tile, over the piece by K.  The number of listed rows is read here.
template <int STEP, bool F16>
struct XentBody {
    const XentArgs &p;
    int rows, m, n;                     // extents of the step's outputs
    __device__ __forceinline__ explicit XentBody(const XentArgs &args) : p(args) {
        rows = __builtin_amdgcn_readfirstlane(listed_count(p));
        m = STEP == 2 ? p.n_count : rows;
        n = STEP == 2 ? p.K : p.n_count;
    }
    __device__ __forceinline__ int total(int bm, int bn) const { return (m + bm - 1) / bm * ((n + bn - 1) / bn); }
    template <class T>
    __device__ __forceinline__ void at(char *lds, int m0, int n0) const {
        if constexpr (STEP == 0) stats_tile<T, F16>(p, rows, lds, m0, n0);
        else if constexpr (STEP == 1) dlogits_tile<T, F16>(p, rows, lds, m0, n0);
        else dw_tile<T, F16>(p, rows, lds, m0, n0);
    }
    template <class T>
    __device__ __forceinline__ void tile(char *lds, int id, int sub) const {
        int tm, tn, m0, n0;
        raster(id, (m + 255) / 256, (n + 255) / 256, tm, tn);
        part_corner<T>(tm, tn, sub, m0, n0);
        if (m0 < m && n0 < n) at<T>(lds, m0, n0);
    }
};

template <int STEP, bool F16>
__global__ void __launch_bounds__(512) xent_mixed_kernel(XentArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[Mixed<STEP != 2>::LDS];
    const XentBody<STEP, F16> body(p);
    Mixed<STEP != 2>::run(body, lds, body.total(256, 256));
}

// Few rows.
template <int STEP, bool F16>
__global__ void __launch_bounds__(Tile32::NT) xent_rows_kernel(XentArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[Tile32::LDS];
    const XentBody<STEP, F16> body(p);
    const int total = body.total(32, 128);
    if ((int)blockIdx.x >= total) return;
    int tm, tn;
    raster(xcd_run(blockIdx.x, total), (body.m + 31) / 32, (body.n + 127) / 128, tm, tn);
    body.template at<Tile32>(lds, 32 * tm, 128 * tn);
}

// dX: sum += P * piece of W, block y of gridDim.y over its share of the piece
// into a sum of its own.  With one share the last piece scales, rounds and
// puts each row in its place; else xent_dx_join_kernel does.
template <class T, bool F16>
__global__ void __launch_bounds__(T::NT) xent_dx_kernel(XentArgs p, int first, int last) {
    __shared__ __attribute__((aligned(16))) char lds[T::LDS];
    const int rows = __builtin_amdgcn_readfirstlane(p.head->rows);
    const int tiles_m = (rows + T::BM - 1) / T::BM, tiles_n = (p.K + T::BN - 1) / T::BN;
    if ((int)blockIdx.x >= tiles_m * tiles_n) return;
    int tm, tn;
    raster(xcd_run(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    const int part = (p.n_count + 64 * (int)gridDim.y - 1) / (64 * (int)gridDim.y) * 64;       // whole K tiles
    const int v0 = min(part * (int)blockIdx.y, p.n_count), v1 = min(v0 + part, p.n_count);
    const Operands16 q = {p.P + 2L * v0, p.W + 2L * (p.n_first + v0) * p.ldw, p.ldp, p.ldw, rows, p.K, v1 - v0};
    f32x4 acc[T::MI][T::NB];
    accumulate16<T, F16, false, false>(q, m0, n0, lds, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool place = last && gridDim.y == 1;
    float *sums = p.sum + (long)blockIdx.y * p.M * p.ldxc;
#pragma unroll
    for (int mi = 0; mi < T::MI; ++mi) {
        const int row = m0 + wave / T::WAVES_N * T::WM + mi * 16 + (lane & 15);
        if (row >= rows) continue;
        float *sum = sums + row * p.ldxc;                     // whole chunks of columns
        char *out = p.dX + 2 * p.map[row] * p.lddx;
        const float scale = p.alpha * p.back[row];
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) {
            const int col = n0 + wave % T::WAVES_N * T::WN + nb * 16 + 4 * (lane >> 4);
            if (col >= p.K) continue;
            f32x4 v = acc[mi][nb];
            if (!first) v += *reinterpret_cast<const f32x4 *>(sum + col);
            if (place) store4<F16, true>(out, col, p.K, 0.f, v * scale);
            else *reinterpret_cast<f32x4 *>(sum + col) = v;
        }
    }
}

// The shares' sums, in order, scaled, rounded and put in place: one block per
// listed row.
template <bool F16>
__global__ void __launch_bounds__(256) xent_dx_join_kernel(XentArgs p, int shares) {
    const int row = blockIdx.x;
    if (row >= p.head->rows) return;
    const float scale = p.alpha * p.back[row];
    char *out = p.dX + 2 * p.map[row] * p.lddx;
    for (int col = 4 * threadIdx.x; col < p.K; col += 1024) {
        const f32x4 v = sum_shares(p.sum + row * p.ldxc + col, p.M * p.ldxc, shares);
        store4<F16, true>(out, col, p.K, 0.f, v * scale);
    }
}

// Bytes of P at most, so that it stays in the Infinity Cache between the
// kernel that writes it and the two that read it.
constexpr long kPieceBytes = 256L << 20;

// (and of the columns of P what the K loop takes as a leading dimension, which
// few rows would pass)
long piece_columns(int M, int N) {
    const long most = std::min(std::max(kPieceBytes / 2 / std::max(M, 1) / 256 * 256, 1024L), kMaxLd16 / 256 * 256L);
    const long pieces = (N + most - 1) / most;
    return ceil_to((N + pieces - 1) / pieces, 256);
}

// Into how many shares the vocabulary (of a piece of `count` columns) is cut
// for dX: its grid of M x K outputs rarely fills the chip and its products are
// long, so as many as fill it, of 512 columns at least (1331 rows of 2048 by
// 50021 columns: 444 us on 128 x 128 tiles unshared, 286 and 15 for the join on
// 256 x 256 in four shares).
int dx_shares(int M, int K, int count) {
    const int bm = M <= 32 ? 32 : M <= 128 ? 128 : 256, bn = M <= 128 ? 128 : 256;
    const long tiles = (M + bm - 1L) / bm * ((K + bn - 1L) / bn), places = M <= 128 ? 512 : 256;
    return (int)std::max(1L, std::min(places / std::max(tiles, 1L), count / 512L));
}

// The workspace, laid out from `base` (null: only its size is wanted).
struct Layout {
    char *base;
    long at = 0;
    char *take(long bytes) {
        char *here = base == nullptr ? nullptr : base + at;
        at += ceil_to(bytes, 256);
        return here;
    }
};

long xent_layout(XentArgs &p, void *workspace, bool grad, char *&Wc) {
    Layout l = {static_cast<char *>(workspace)};
    p.ldxc = ceil_to(p.K, 8);
    p.take_x = chunk_rows(p.X, p.ldx, p.K);
    p.head = reinterpret_cast<XentHead *>(l.take(sizeof(XentHead)));
    p.map = reinterpret_cast<int *>(l.take(4L * p.M));
    p.label = reinterpret_cast<int *>(l.take(4L * p.M));
    const long segments = p.M > kOnePass ? (p.M + kSegment - 1) / kSegment : 0;
    p.seg_rows = reinterpret_cast<int *>(l.take(4 * segments));
    p.seg_max = reinterpret_cast<float *>(l.take(4 * segments));
    p.Xc = l.take(2L * p.M * p.ldxc);
    Wc = chunk_rows(p.W, p.ldw, p.K) ? nullptr : l.take(2L * p.N * p.ldxc);
    if (!grad) {
        p.tlogit = reinterpret_cast<float *>(l.take(4L * p.M));
        p.part = reinterpret_cast<float2 *>(l.take(8L * p.M * ((p.N + 127L) / 128)));
    } else {
        p.g = reinterpret_cast<float *>(l.take(4L * p.M));
        p.lsec = reinterpret_cast<float *>(l.take(4L * p.M));
        p.back = reinterpret_cast<float *>(l.take(4L * p.M));
        p.down = reinterpret_cast<float *>(l.take(4L * p.M));
        p.ldp = piece_columns(p.M, p.N);
        p.P = l.take(2L * p.M * p.ldp);
        const int shares = dx_shares(p.M, p.K, (int)std::min((long)p.N, p.ldp));
        p.sum = p.ldp < p.N || shares > 1 ? reinterpret_cast<float *>(l.take(4L * shares * p.M * p.ldxc)) : nullptr;
    }
    return l.at;
}

int check(int dtype, int M, int N, int K, int ldx, int ldw) {
    if (dtype != SGEMM_DTYPE_BF16 && dtype != SGEMM_DTYPE_F16) return SGEMM_STATUS_INVALID_DTYPE;
    // (the vocabulary must hold a column for the sums to have a term)
    if (M < 0 || N < 1 || K < 0 || ldx < std::max(K, 1) || ldw < std::max(K, 1) || K > kMaxLd16 ||
        M > (1 << 24) || N > (1 << 30))
        return SGEMM_STATUS_INVALID_DIM;
    // (the tiles of the logits, of dW and of dX; few rows take smaller ones, of which there are fewer)
    auto fits = [](long m, long n) { return launch_fits(mixed_grid((m + 255) / 256 * ((n + 255) / 256)), 512); };
    if (!fits(M, N) || !fits(N, K) || !fits(M, K)) return SGEMM_STATUS_INVALID_DIM;
    return SGEMM_STATUS_OK;
}

bool scratch_ok(long need, const void *workspace, long long bytes) {
    return workspace != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(workspace) & 15) == 0;
}

unsigned tiles(long m, long n, int bm, int bn) { return (unsigned)((m + bm - 1) / bm * ((n + bn - 1) / bn)); }

template <bool GRAD>
hipError_t launch_compact(const XentArgs &p, hipStream_t s) {
    if (p.M > kOnePass) {
        const hipError_t e = launch_k(xent_segments_kernel<GRAD>, dim3((p.M + kSegment - 1) / kSegment), dim3(256), s, p);
        if (e != hipSuccess) return e;
    }
    // (M == 0: one block, which finds no row)
    return launch_k(xent_compact_kernel<GRAD>, dim3(std::max((p.M + kCompactRows - 1) / kCompactRows, 1)), dim3(256), s, p);
}

template <int STEP>
hipError_t launch_mixed(const XentArgs &p, long m, long n, bool f16, hipStream_t s) {
    const dim3 grid((unsigned)mixed_grid(tiles(m, n, 256, 256)));
    return f16 ? launch_k(xent_mixed_kernel<STEP, true>, grid, dim3(512), s, p)
               : launch_k(xent_mixed_kernel<STEP, false>, grid, dim3(512), s, p);
}

// Steps 0 and 1, on a tile of 32 rows (bound by the bytes of W) or large ones.
template <int STEP>
hipError_t launch_logits(const XentArgs &p, bool f16, hipStream_t s) {
    if (p.M > 32) return launch_mixed<STEP>(p, p.M, p.n_count, f16, s);
    const dim3 grid(tiles(p.M, p.n_count, 32, 128));
    return f16 ? launch_k(xent_rows_kernel<STEP, true>, grid, dim3(Tile32::NT), s, p)
               : launch_k(xent_rows_kernel<STEP, false>, grid, dim3(Tile32::NT), s, p);
}

template <class T>
hipError_t launch_dx(const XentArgs &p, int shares, int first, int last, bool f16, hipStream_t s) {
    const dim3 grid(tiles(p.M, p.K, T::BM, T::BN), shares);
    return f16 ? launch_k(xent_dx_kernel<T, true>, grid, dim3(T::NT), s, p, first, last)
               : launch_k(xent_dx_kernel<T, false>, grid, dim3(T::NT), s, p, first, last);
}

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

long long sgemm_lowp_xent_workspace(int M, int N, int K, const void *X, int ldx, const void *W, int ldw, int grad) {
    const int st = check(SGEMM_DTYPE_BF16, M, N, K, ldx, ldw);
    if (st != SGEMM_STATUS_OK) return st;
    XentArgs p = {};
    p.X = static_cast<const char *>(X);
    p.W = static_cast<const char *>(W);
    p.ldx = ldx;
    p.ldw = ldw;
    p.M = M;
    p.N = N;
    p.K = K;
    char *Wc;
    return M == 0 && !grad ? 0 : xent_layout(p, nullptr, grad != 0, Wc);
}

int sgemm_lowp_xent(int dtype, int M, int N, int K, float alpha, const void *X, int ldx, const void *W, int ldw,
                    const long long *target, long long ignore_index, float *loss, float *lse, void *workspace,
                    long long workspace_bytes, void *stream) {
    const int st = check(dtype, M, N, K, ldx, ldw);
    if (st != SGEMM_STATUS_OK) return st;
    if (M == 0) return SGEMM_STATUS_OK;
    if (target == nullptr || loss == nullptr || lse == nullptr || (K > 0 && (X == nullptr || W == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    XentArgs p = {};
    p.X = static_cast<const char *>(X);
    p.W = static_cast<const char *>(W);
    p.ldx = ldx;
    p.ldw = ldw;
    p.M = M;
    p.N = p.n_count = N;
    p.K = K;
    p.alpha = alpha;
    p.target = target;
    p.ignore = ignore_index;
    p.loss = loss;
    p.lse = lse;
    char *Wc;
    if (!scratch_ok(xent_layout(p, nullptr, false, Wc), workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    xent_layout(p, workspace, false, Wc);
    const bool f16 = dtype == SGEMM_DTYPE_F16;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    // (Rows do not meet in the forward pass, so listing the ones that count
    // only saves work; for few rows of an aligned X it costs more: 17 x 32000 x
    // 1024 20.1 us with it, 16.8 without.)
    p.direct = M <= 32 && p.take_x;
    hipError_t e = p.direct ? hipSuccess : launch_compact<false>(p, s);
    if (e == hipSuccess && Wc != nullptr) {
        e = pad_rows(W, ldw, 0, 1, N, K, Wc, s);
        p.W = Wc;
        p.ldw = p.ldxc;
    }
    if (e == hipSuccess) e = launch_logits<0>(p, f16, s);
    if (e == hipSuccess) e = launch_k(xent_join_kernel, dim3((M + 15) / 16), dim3(1024), s, p, (N + 127) / 128);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_lowp_xent_grad(int dtype, int M, int N, int K, float alpha, const void *X, int ldx, const void *W, int ldw,
                         const long long *target, long long ignore_index, const float *lse, const float *dloss,
                         int dloss_stride, void *dX, int lddx, void *dW, int lddw, void *workspace,
                         long long workspace_bytes, void *stream) {
    const int st = check(dtype, M, N, K, ldx, ldw);
    if (st != SGEMM_STATUS_OK) return st;
    if (dloss_stride < 0 || (dX != nullptr && lddx < std::max(K, 1)) || (dW != nullptr && lddw < std::max(K, 1)))
        return SGEMM_STATUS_INVALID_DIM;
    if (K == 0 || (dX == nullptr && dW == nullptr) || (M == 0 && dW == nullptr)) return SGEMM_STATUS_OK;
    if (W == nullptr || (M > 0 && (X == nullptr || target == nullptr || lse == nullptr || dloss == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    XentArgs p = {};
    p.X = static_cast<const char *>(X);
    p.W = static_cast<const char *>(W);
    p.ldx = ldx;
    p.ldw = ldw;
    p.M = M;
    p.N = N;
    p.K = K;
    p.alpha = alpha;
    p.target = target;
    p.ignore = ignore_index;
    p.lse_in = lse;
    p.dloss = dloss;
    p.dloss_stride = dloss_stride;
    p.dX = static_cast<char *>(dX);
    p.dW = static_cast<char *>(dW);
    p.lddx = lddx;
    p.lddw = lddw;
    char *Wc;
    if (!scratch_ok(xent_layout(p, nullptr, true, Wc), workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    xent_layout(p, workspace, true, Wc);
    const bool f16 = p.f16 = dtype == SGEMM_DTYPE_F16;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = launch_compact<true>(p, s);
    if (e == hipSuccess && Wc != nullptr) {
        e = pad_rows(W, ldw, 0, 1, N, K, Wc, s);
        p.W = Wc;
        p.ldw = p.ldxc;
    }
    const int shares = dx_shares(M, K, (int)std::min((long)N, p.ldp));
    for (p.n_first = 0; p.n_first < N && e == hipSuccess; p.n_first += (int)p.ldp) {
        p.n_count = (int)std::min((long)N - p.n_first, p.ldp);
        const int first = p.n_first == 0, last = p.n_first + p.n_count == N;
        if (M > 0) e = launch_logits<1>(p, f16, s);
        if (e == hipSuccess && M > 0 && dX != nullptr)
            e = M <= 32    ? launch_dx<Tile32>(p, shares, first, last, f16, s)
                : M <= 128 ? launch_dx<Tile128>(p, shares, first, last, f16, s)
                           : launch_dx<Tile256>(p, shares, first, last, f16, s);
        if (e == hipSuccess && M > 1 && dW != nullptr && f16 && dloss_stride != 0) {     // (else no row is apart)
            const int across = std::min(M, 1024), along = std::min((p.n_count + 2047) / 2048, (1023 + across) / across);
            e = launch_k(xent_rescale_kernel, dim3(across, along), dim3(256), s, p);
        }
        if (e == hipSuccess && dW != nullptr) e = launch_mixed<2>(p, p.n_count, K, f16, s);
    }
    if (e == hipSuccess && M > 0 && dX != nullptr && shares > 1)
        e = f16 ? launch_k(xent_dx_join_kernel<true>, dim3(M), dim3(256), s, p, shares)
                : launch_k(xent_dx_join_kernel<false>, dim3(M), dim3(256), s, p, shares);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

}  // extern "C"

// Tokens sorted by expert and back: T tokens of `picks` experts each, so
// n = T * picks assignments i = t * picks + j, whose key is the expert, or
// `groups` where that is none of 0 .. groups - 1.
//
//   sort     place of i = #{keys below its own} + #{equal keys before it}, a
//            stable counting sort; token rows are copied to their places
//     sort_few_kernel     every place counted on its own; and the copies
//     sort_count_kernel, sort_place_kernel, sort_copy_kernel
//   combine  out[t] = sum_j weights[t][j] * Y[place of (t, j)], in FP32, j in order
//     combine_kernel
//   grad     dY[place of (t, j)] = weights[t][j] * D[t],
//            dweights[t][j] = <D[t], Y[place of (t, j)]>, summed in FP32
//     combine_grad_kernel
//
// All but the counting is bound by the rows' bytes.  A token's row is read once
// and written to (or read with) all of its places, in 16-byte pieces whatever
// the rows' alignment (this chip takes such accesses at any byte), by 16, 64 or
// 256 lanes, as wide as a row is.
#include <algorithm>
#include <type_traits>

#include "sgemm_rows.hpp"

namespace sgemm_mi355x {

namespace {

struct SortArgs {
    const char *X;
    char *rows;
    const float *x_scales;
    float *row_scales;
    const void *experts;
    int *offsets, *position, *source, *counts;
    long ldx, ldr, lde;                     // bytes; bytes; elements
    int T, picks, groups, n;
    int width;                              // bytes of a row
    int wide;                               // experts in 64 bits
    int chunk;                              // assignments per workgroup of the counting kernels
    int lanes;                              // per token in the copies
    __device__ __forceinline__ int key(int i) const {
        long at = i;
        if (lde != picks) {
            const int t = (unsigned)i / (unsigned)picks;
            at = t * lde + (i - t * picks);
        }
        const long e = wide ? static_cast<const long long *>(experts)[at] : static_cast<const int *>(experts)[at];
        return (unsigned long)e < (unsigned long)groups ? (int)e : groups;
    }
};

// One 16-byte piece of a row of `width` bytes, at byte c < width.
__device__ __forceinline__ i32x4 load_piece(const char *row, int c, int width) {
    i32x4 v = {0, 0, 0, 0};
    if (c + 16 <= width) __builtin_memcpy(&v, row + c, 16);
    else
        for (int e = 0; c + e < width; ++e) v[e >> 2] |= (int)((unsigned)(unsigned char)row[c + e] << (8 * (e & 3)));
    return v;
}

__device__ __forceinline__ void store_piece(char *row, int c, int width, i32x4 v) {
    if (c + 16 <= width) __builtin_memcpy(row + c, &v, 16);
    else
        for (int e = 0; c + e < width; ++e) row[c + e] = (char)((unsigned)v[e >> 2] >> (8 * (e & 3)));
}

// Token t's row to its places; of the rows t * picks .. + picks - 1 those of no
// group become zeros.  `lane` of `lanes` lanes.
__device__ __forceinline__ void copy_token(const SortArgs &p, int t, const int *places, int kept, int lane) {
    const char *x = p.X + t * p.ldx;
    const int first = t * p.picks;
    for (int c = 16 * lane; c < p.width; c += 16 * p.lanes) {
        const i32x4 v = load_piece(x, c, p.width);
        for (int j = 0; j < p.picks; ++j) {
            const int at = places[j];
            if (at >= 0) store_piece(p.rows + at * p.ldr, c, p.width, v);
            if (first + j >= kept) store_piece(p.rows + (first + j) * p.ldr, c, p.width, i32x4{0, 0, 0, 0});
        }
    }
    if (p.row_scales) {
        for (int j = lane; j < p.picks; j += p.lanes) {
            if (places[j] >= 0) p.row_scales[places[j]] = p.x_scales[t];
            if (first + j >= kept) p.row_scales[first + j] = 0.f;
        }
    }
}

// Up to kFew assignments, in one launch: each workgroup holds all keys in LDS
// and counts for itself the places of its tokens' assignments (a wave each)
// and the bounds of some groups, then copies its tokens' rows.  1024 assignments
// 5.3 us where the three kernels below take 6.9, but 4096 11 to 18.
constexpr int kFew = 2048;

__global__ void __launch_bounds__(256) sort_few_kernel(SortArgs p) {
    __shared__ __attribute__((aligned(16))) int keys[kFew + 256];
    __shared__ int places[kFew], kept;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, upto = (p.n + 255) & ~255;
    for (int i = threadIdx.x; i < upto; i += 256) keys[i] = i < p.n ? p.key(i) : 0x7fffffff;   // (neither below a key nor one)
    __syncthreads();
    auto below = [&](int key, int self) {   // keys below `key`, and equal ones before assignment `self`
        int count = 0;
#pragma unroll 4
        for (int i = 4 * lane; i < upto; i += 256) {
            const i32x4 k = *reinterpret_cast<const i32x4 *>(keys + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) count += k[e] < key || (k[e] == key && i + e < self);
        }
        return wave_sum(count);
    };
    // the bounds: a thread each where a thread's count is short, else a wave each
    if (p.n <= 64) {
        for (int g = blockIdx.x * 256 + threadIdx.x; g <= p.groups; g += gridDim.x * 256) {
            int count = 0;
            for (int i = 0; i < p.n; ++i) count += keys[i] < g;
            p.offsets[g] = count;
        }
    } else {
        for (int g = blockIdx.x * 4 + wave; g <= p.groups; g += gridDim.x * 4) {
            const int count = below(g, 0);
            if (lane == 0) p.offsets[g] = count;
        }
    }
    if (wave == 0) {
        const int count = below(p.groups, 0);
        if (lane == 0) kept = count;
    }
    // tokens first .. last - 1 are this workgroup's
    const int first = (int)((long)p.T * blockIdx.x / gridDim.x), last = (int)((long)p.T * (blockIdx.x + 1) / gridDim.x);
    for (int i = first * p.picks + wave; i < last * p.picks; i += 4) {
        const int key = keys[i], at = below(key, i), place = key < p.groups ? at : -1;
        if (lane == 0) {
            p.position[i] = place;
            p.source[at] = place < 0 ? -1 : i;
            places[i] = place;
        }
    }
    if (p.rows == nullptr && p.row_scales == nullptr) return;
    __syncthreads();
    const int per = 256 / p.lanes;
    for (int t = first + threadIdx.x / p.lanes; t < last; t += per)
        copy_token(p, t, places + t * p.picks, kept, threadIdx.x & (p.lanes - 1));
}

// More of them: `blocks` workgroups take `chunk` assignments each (65536
// assignments to 128 groups: 4.7 us, and 6.8 for the places).
//
// counts[block][key]: how often each key is among the block's assignments.
constexpr int kMaxSortGroups = 4096, kMaxBins = kMaxSortGroups + 1;

__global__ void __launch_bounds__(256) sort_count_kernel(SortArgs p) {
    __shared__ int table[kMaxBins];
    const int bins = p.groups + 1;
    for (int g = threadIdx.x; g < bins; g += 256) table[g] = 0;
    __syncthreads();
    const long first = (long)blockIdx.x * p.chunk, last = min(first + p.chunk, (long)p.n);
    for (long i = first + threadIdx.x; i < last; i += 256) atomicAdd(&table[p.key((int)i)], 1);
    __syncthreads();
    for (int g = threadIdx.x; g < bins; g += 256) p.counts[(long)blockIdx.x * bins + g] = table[g];
}

// The places of a block's assignments: where its keys' rows begin follows from
// all blocks' counts, and within the block each of the W waves takes a run of
// assignments in order, 64 at a time, whose equal keys find each other by the
// bits of the key.
template <int W, int BINS>
__global__ void __launch_bounds__(64 * W) sort_place_kernel(SortArgs p) {
    __shared__ int table[W][BINS], start[BINS], before[BINS];
    constexpr int NT = 64 * W;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int bins = p.groups + 1, blocks = gridDim.x, block = blockIdx.x;
    for (int g = threadIdx.x; g < bins; g += NT) {
        start[g] = before[g] = 0;
        for (int w = 0; w < W; ++w) table[w][g] = 0;
    }
    __syncthreads();
    // all blocks' counts, and those of the blocks before: where there are fewer
    // keys than threads, several threads share a key's blocks
    const int slices = max(NT / bins, 1);
    for (int u = threadIdx.x; u < bins * slices; u += NT) {
        const int g = u % bins;
        int all = 0, less = 0;
#pragma unroll 8
        for (int b = u / bins; b < blocks; b += slices) {
            const int c = p.counts[(long)b * bins + g];
            all += c;
            less += b < block ? c : 0;
        }
        atomicAdd(&start[g], all);
        atomicAdd(&before[g], less);
    }
    const long first = (long)block * p.chunk, end = min(first + p.chunk, (long)p.n);
    const long run = (p.chunk + NT - 1) / NT * 64, from = min(first + wave * run, end), to = min(from + run, end);
    for (long i = from + lane; i < to; i += 64) atomicAdd(&table[wave][p.key((int)i)], 1);
    __syncthreads();
    if (wave == 0) {                        // start: sums of the keys below
        int sum = 0;
        for (int g0 = 0; g0 < bins; g0 += 64) {
            const int g = g0 + lane, mine = g < bins ? start[g] : 0;
            int upto = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int other = __shfl_up(upto, d);
                if (lane >= d) upto += other;
            }
            if (g < bins) start[g] = sum + upto - mine;
            sum += __shfl(upto, 63);
        }
    }
    __syncthreads();
    for (int g = threadIdx.x; g < bins; g += NT) {
        int at = start[g] + before[g];
        for (int w = 0; w < W; ++w) {
            const int c = table[w][g];
            table[w][g] = at;
            at += c;
        }
        if (block == 0) p.offsets[g] = start[g];
    }
    __syncthreads();
    volatile int *mine = table[wave];
    const int bits = 32 - __builtin_clz(p.groups | 1);
    for (long i0 = from; i0 < to; i0 += 64) {
        const bool live = i0 + lane < to;
        const int i = live ? (int)i0 + lane : 0;
        const int key = live ? p.key(i) : 0;
        unsigned long same = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const unsigned long set = __ballot(key >> b & 1);
            same &= key >> b & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ul << lane) - 1)), count = __popcll(same);
        int at = 0;
        if (live) at = mine[key] + rank;
        __builtin_amdgcn_wave_barrier();
        if (live && rank == count - 1) mine[key] = at + 1;
        __builtin_amdgcn_wave_barrier();
        if (live) {
            const bool kept = key < p.groups;
            p.position[i] = kept ? at : -1;
            p.source[at] = kept ? i : -1;
        }
    }
}

// 8192 rows of 4096 in BF16 to eight places each: 104 us, 5.8 TB/s.
__global__ void __launch_bounds__(256) sort_copy_kernel(SortArgs p) {
    const int per = 256 / p.lanes, kept = p.offsets[p.groups];
    for (long t = (long)blockIdx.x * per + threadIdx.x / p.lanes; t < p.T; t += (long)gridDim.x * per)
        copy_token(p, (int)t, p.position + t * p.picks, kept, threadIdx.x & (p.lanes - 1));
}

// ---------------------------------------------------------------------------

struct CombineArgs {
    const char *Y, *D;                      // [n][H], [T][H]
    char *out;                              // combine: [T][H]; grad: dY [n][H]
    const int *offsets, *position;
    const char *weights;                    // [T][picks], NULL: 1
    char *dweights;                         // [T][picks]
    long ldy, ldd, ldo, ldw;                // elements
    int T, picks, groups, H, n, dtype_w, lanes;
    __device__ __forceinline__ float weight(int t, int j) const {
        if (weights == nullptr) return 1.f;
        const long at = t * ldw + j;
        if (dtype_w == SGEMM_DTYPE_F32) return reinterpret_cast<const float *>(weights)[at];
        const unsigned short bits = reinterpret_cast<const unsigned short *>(weights)[at];
        return dtype_w == SGEMM_DTYPE_F16 ? widen16<true>(bits) : widen16<false>(bits);
    }
    // The place of token t's pick j, -1 for none (whatever the array holds).
    __device__ __forceinline__ int place(int t, int j) const {
        const int at = position[(long)t * picks + j];
        return (unsigned)at < (unsigned)n ? at : -1;
    }
};

constexpr int kBf16Row = SGEMM_DTYPE_BF16, kF16Row = SGEMM_DTYPE_F16, kF32Row = SGEMM_DTYPE_F32;

// Eight values of a row of elements from column c on.
template <int DTYPE>
struct Row8 {
    static constexpr int E = DTYPE == kF32Row ? 4 : 2, WORDS = 2 * E;
    int w[WORDS];
    __device__ __forceinline__ void load(const char *base, long row, long ld, int c, int H) {
        const char *at = base + (row * ld + c) * E;
        if (c + 8 <= H) {
            __builtin_memcpy(w, at, 8 * E);
        } else {
            for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c + e >= H) break;
                if constexpr (E == 4) w[e] = reinterpret_cast<const int *>(at)[e];
                else w[e >> 1] |= (int)((unsigned)reinterpret_cast<const unsigned short *>(at)[e] << (16 * (e & 1)));
            }
        }
    }
    __device__ __forceinline__ float at(int e) const {
        if constexpr (E == 4) return __int_as_float(w[e]);
        return widen16<DTYPE == kF16Row>((unsigned short)((unsigned)w[e >> 1] >> (16 * (e & 1))));
    }
};

template <int DTYPE>
__device__ __forceinline__ void store8(char *base, long row, long ld, int c, int H, const float (&v)[8]) {
    constexpr int E = DTYPE == kF32Row ? 4 : 2;
    char *at = base + row * ld * E;
    if (E == 2 && c + 8 <= H) {             // both halves in one access
        const i32x2 a = round16<DTYPE == kF16Row>(f32x4{v[0], v[1], v[2], v[3]}), b = round16<DTYPE == kF16Row>(f32x4{v[4], v[5], v[6], v[7]});
        const i32x4 o = {a[0], a[1], b[0], b[1]};
        __builtin_memcpy(at + c * 2l, &o, 16);
        return;
    }
    store4<DTYPE == kF16Row, E == 2>(at, c, H, 0.f, f32x4{v[0], v[1], v[2], v[3]});
    if (c + 4 < H) store4<DTYPE == kF16Row, E == 2>(at, c + 4, H, 0.f, f32x4{v[4], v[5], v[6], v[7]});
}

// A piece of a token's row per `lanes` lanes and turn, with PICKS rows of Y in
// flight.  8192 x 8 rows of 4096 in BF16 122 us, 4.9 TB/s (with four rows in flight
// and a token's pieces one after another 141; 512 x 8 rows of 7168 23 and 34).  The
// grid is sized by the tokens: where those are few their pieces follow one another
// (16 x 8 rows of 7168 12 us).
template <int YT, int OT>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs p) {
    constexpr int PICKS = YT == kF32Row ? 4 : 8;
    const int lane = threadIdx.x & (p.lanes - 1), per = 256 / p.lanes, cuts = (p.H + 8 * p.lanes - 1) / (8 * p.lanes);
    for (long u = (long)blockIdx.x * per + threadIdx.x / p.lanes; u < (long)p.T * cuts; u += (long)gridDim.x * per) {
        const int t = (int)(u / cuts), c = 8 * (lane + (int)(u - (long)t * cuts) * p.lanes);
        if (c >= p.H) continue;
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int j0 = 0; j0 < p.picks; j0 += PICKS) {
            Row8<YT> y[PICKS];
            int at[PICKS];
            float w[PICKS];
#pragma unroll
            for (int j = 0; j < PICKS; ++j) {
                at[j] = -1;
                if (j0 + j < p.picks) {
                    at[j] = p.place(t, j0 + j);
                    w[j] = p.weight(t, j0 + j);
                }
            }
#pragma unroll
            for (int j = 0; j < PICKS; ++j)
                if (at[j] >= 0) y[j].load(p.Y, at[j], p.ldy, c, p.H);
#pragma unroll
            for (int j = 0; j < PICKS; ++j) {
                if (at[j] < 0) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += w[j] * y[j].at(e);
            }
        }
        store8<OT>(p.out, t, p.ldo, c, p.H, sum);
    }
}

// YT: the type of Y and dY, DT: of D.  PICKS rows at a time, whose dot products
// need all lanes of a token.  16384 x 2 rows of 4096 in BF16: 136 us, 4.9 TB/s.
template <int YT, int DT>
__global__ void __launch_bounds__(256) combine_grad_kernel(CombineArgs p) {
    constexpr int PICKS = 4;
    __shared__ float part[4][PICKS];
    const int lane = threadIdx.x & (p.lanes - 1), per = 256 / p.lanes, kept = p.offsets[p.groups];
    const float none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // (every thread of a workgroup makes the same number of turns: barriers within)
    for (long t0 = (long)blockIdx.x * per; t0 < p.T; t0 += (long)gridDim.x * per) {
        const long t = t0 + threadIdx.x / p.lanes;
        const bool live = t < p.T;
        for (int j0 = 0; j0 < p.picks; j0 += PICKS) {
            int at[PICKS];
            float w[PICKS], dot[PICKS];
#pragma unroll
            for (int j = 0; j < PICKS; ++j) {
                const bool in = live && j0 + j < p.picks;
                at[j] = in ? p.place((int)t, j0 + j) : -1;
                w[j] = in ? p.weight((int)t, j0 + j) : 0.f;
                dot[j] = 0.f;
            }
            if (live) {
                for (int c = 8 * lane; c < p.H; c += 8 * p.lanes) {
                    Row8<DT> d;
                    Row8<YT> y[PICKS];
                    d.load(p.D, t, p.ldd, c, p.H);
                    if (p.dweights) {
#pragma unroll
                        for (int j = 0; j < PICKS; ++j)
                            if (at[j] >= 0) y[j].load(p.Y, at[j], p.ldy, c, p.H);
                    }
#pragma unroll
                    for (int j = 0; j < PICKS; ++j) {
                        if (at[j] >= 0) {
                            if (p.dweights) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) dot[j] += d.at(e) * y[j].at(e);
                            }
                            if (p.out) {
                                float v[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = w[j] * d.at(e);
                                store8<YT>(p.out, at[j], p.ldo, c, p.H, v);
                            }
                        }
                        // of rows t * picks .. + picks - 1 those of no group are zeros
                        const long row = t * p.picks + j0 + j;
                        if (p.out && j0 + j < p.picks && row >= kept) store8<YT>(p.out, row, p.ldo, c, p.H, none);
                    }
                }
            }
            if (p.dweights == nullptr) continue;
#pragma unroll
            for (int j = 0; j < PICKS; ++j)
                for (int d = min(p.lanes, 64) / 2; d; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
            if (p.lanes > 64) {
                if ((threadIdx.x & 63) == 0) {
#pragma unroll
                    for (int j = 0; j < PICKS; ++j) part[threadIdx.x >> 6][j] = dot[j];
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < PICKS; ++j) dot[j] = part[0][j] + part[1][j] + part[2][j] + part[3][j];
                __syncthreads();
            }
            if (live && lane == 0) {
#pragma unroll
                for (int j = 0; j < PICKS; ++j) {
                    if (j0 + j >= p.picks) break;
                    const long to = t * p.picks + j0 + j;
                    if (p.dtype_w == SGEMM_DTYPE_F32) reinterpret_cast<float *>(p.dweights)[to] = dot[j];
                    else {
                        const f32x4 v = {dot[j], dot[j], dot[j], dot[j]};
                        reinterpret_cast<unsigned short *>(p.dweights)[to] =
                            (unsigned short)(p.dtype_w == SGEMM_DTYPE_F16 ? round16<true>(v)[0] : round16<false>(v)[0]);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------

int lanes_for(long pieces) { return pieces <= 16 ? 16 : pieces <= 64 ? 64 : 256; }

// One workgroup per 256 / lanes tokens, as many as a launch takes.
unsigned token_blocks(int T, int lanes) { return (unsigned)std::min((T + 256L / lanes - 1) / (256 / lanes), 1L << 20); }

// Workgroups of the counting kernels: 512 assignments each, but no more than
// 256 (every one reads all others' counts), and 2^16 counts in all.
int sort_blocks(int n, int groups) {
    return (int)std::max(1L, std::min({(n + 511L) / 512, 256L, std::max(8L, 65536L / (groups + 1))}));
}

bool float_type(int d) { return d == SGEMM_DTYPE_BF16 || d == SGEMM_DTYPE_F16 || d == SGEMM_DTYPE_F32; }

int size_of(int d) { return d == SGEMM_DTYPE_I8 ? 1 : d == SGEMM_DTYPE_F32 ? 4 : 2; }

bool pair_ok(int y, int other) { return float_type(y) && float_type(other) && (y == other || y == SGEMM_DTYPE_F32 || other == SGEMM_DTYPE_F32); }

bool sizes_ok(int T, int picks, int H) { return T >= 0 && picks >= 0 && H >= 0 && H <= (1 << 28) && (long)T * picks < (1L << 31) - 1; }

// f(type of Y, the other type)
template <class F>
hipError_t by_pair(int y, int other, F &&f) {
    if (y == SGEMM_DTYPE_F32)
        return other == SGEMM_DTYPE_F32 ? f(IntC<kF32Row>{}, IntC<kF32Row>{}) : other == SGEMM_DTYPE_BF16 ? f(IntC<kF32Row>{}, IntC<kBf16Row>{}) : f(IntC<kF32Row>{}, IntC<kF16Row>{});
    if (y == SGEMM_DTYPE_BF16) return other == y ? f(IntC<kBf16Row>{}, IntC<kBf16Row>{}) : f(IntC<kBf16Row>{}, IntC<kF32Row>{});
    return other == y ? f(IntC<kF16Row>{}, IntC<kF16Row>{}) : f(IntC<kF16Row>{}, IntC<kF32Row>{});
}

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

long long sgemm_grouped_sort_workspace(int T, int picks, int groups) {
    if (!sizes_ok(T, picks, 0) || groups < 0 || groups > kMaxSortGroups) return SGEMM_STATUS_INVALID_DIM;
    const int n = T * picks;
    return n <= kFew ? 0 : ceil_to(4L * sort_blocks(n, groups) * (groups + 1), 16);
}

int sgemm_grouped_sort(int dtype, int T, int picks, int groups, int H, const void *X, int ldx, const float *x_scales,
                       const void *experts, int lde, int expert_bytes, int *offsets, int *position, int *source, void *rows,
                       int ldr, float *row_scales, void *workspace, long long workspace_bytes, void *stream) {
    if ((!float_type(dtype) && dtype != SGEMM_DTYPE_I8) || (expert_bytes != 4 && expert_bytes != 8)) return SGEMM_STATUS_INVALID_DTYPE;
    if (!sizes_ok(T, picks, H) || groups < 0 || groups > kMaxSortGroups || lde < picks) return SGEMM_STATUS_INVALID_DIM;
    if (rows != nullptr && (ldx < std::max(H, 1) || ldr < std::max(H, 1))) return SGEMM_STATUS_INVALID_DIM;
    const int n = T * picks, size = size_of(dtype);
    if (offsets == nullptr || (n > 0 && (experts == nullptr || position == nullptr || source == nullptr))) return SGEMM_STATUS_NULL_POINTER;
    // (rows of no columns have scales to bring, and no address)
    const bool copies = n > 0 && (rows != nullptr || (dtype == SGEMM_DTYPE_I8 && H == 0 && row_scales != nullptr));
    if (copies && ((H > 0 && X == nullptr) || (dtype == SGEMM_DTYPE_I8 && (x_scales == nullptr || row_scales == nullptr))))
        return SGEMM_STATUS_NULL_POINTER;
    if (!copies) rows = nullptr, row_scales = nullptr;      // (X may be NULL)
    const long long need = sgemm_grouped_sort_workspace(T, picks, groups);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15))) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SortArgs p = {static_cast<const char *>(X), static_cast<char *>(rows), x_scales, dtype == SGEMM_DTYPE_I8 ? row_scales : nullptr, experts,
                  offsets, position, source, static_cast<int *>(workspace), (long)ldx * size, (long)ldr * size, lde, T, picks, groups, n,
                  H * size, expert_bytes == 8, 0, lanes_for((H * (long)size + 15) / 16)};
    if (n <= kFew) {
        const hipError_t e = launch_k(sort_few_kernel, dim3((unsigned)std::min(std::max(T, 1), 512)), dim3(256), s, p);
        return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
    }
    const int blocks = sort_blocks(n, groups);
    p.chunk = (int)((n + (long)blocks - 1) / blocks);
    hipError_t e = launch_k(sort_count_kernel, dim3((unsigned)blocks), dim3(256), s, p);
    if (e == hipSuccess)
        e = groups + 1 <= 2048 ? launch_k(sort_place_kernel<16, 2048>, dim3((unsigned)blocks), dim3(1024), s, p)
                               : launch_k(sort_place_kernel<4, kMaxBins>, dim3((unsigned)blocks), dim3(256), s, p);
    if (e == hipSuccess && copies) e = launch_k(sort_copy_kernel, dim3(token_blocks(T, p.lanes)), dim3(256), s, p);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_grouped_combine(int dtype, int dtype_out, int T, int picks, int H, const void *Y, int ldy, const int *position,
                          const void *weights, int ldw, int dtype_w, void *out, int ldo, void *stream) {
    if (!pair_ok(dtype, dtype_out) || (weights != nullptr && !float_type(dtype_w))) return SGEMM_STATUS_INVALID_DTYPE;
    if (!sizes_ok(T, picks, H) || ldy < std::max(H, 1) || ldo < std::max(H, 1) || (weights != nullptr && ldw < picks)) return SGEMM_STATUS_INVALID_DIM;
    if (T == 0 || H == 0) return SGEMM_STATUS_OK;
    if (out == nullptr || (picks > 0 && (Y == nullptr || position == nullptr))) return SGEMM_STATUS_NULL_POINTER;
    const CombineArgs p = {static_cast<const char *>(Y), nullptr, static_cast<char *>(out), nullptr, position, static_cast<const char *>(weights), nullptr,
                           ldy, 0, ldo, ldw, T, picks, 0, H, T * picks, dtype_w, lanes_for((H + 7L) / 8)};
    const hipError_t e = by_pair(dtype, dtype_out, [&](auto y, auto o) {
        return launch_k(combine_kernel<decltype(y)::value, decltype(o)::value>, dim3(token_blocks(p.T, p.lanes)), dim3(256),
                        reinterpret_cast<hipStream_t>(stream), p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_grouped_combine_grad(int dtype, int dtype_d, int T, int picks, int groups, int H, const void *D, int ldd, const void *Y,
                               int ldy, const int *offsets, const int *position, const void *weights, int ldw, int dtype_w,
                               void *dY, int lddy, void *dweights, void *stream) {
    if (!pair_ok(dtype, dtype_d) || ((weights != nullptr || dweights != nullptr) && !float_type(dtype_w))) return SGEMM_STATUS_INVALID_DTYPE;
    if (!sizes_ok(T, picks, H) || groups < 0 || ldd < std::max(H, 1)) return SGEMM_STATUS_INVALID_DIM;
    if ((dweights != nullptr && ldy < std::max(H, 1)) || (dY != nullptr && lddy < std::max(H, 1)) || (weights != nullptr && ldw < picks)) return SGEMM_STATUS_INVALID_DIM;
    if (T == 0 || picks == 0 || (dY == nullptr && dweights == nullptr)) return SGEMM_STATUS_OK;
    if (offsets == nullptr || position == nullptr || (H > 0 && (D == nullptr || (dweights != nullptr && Y == nullptr)))) return SGEMM_STATUS_NULL_POINTER;
    const CombineArgs p = {static_cast<const char *>(Y), static_cast<const char *>(D), static_cast<char *>(dY), offsets, position,
                           static_cast<const char *>(weights), static_cast<char *>(dweights), ldy, ldd, lddy, ldw, T, picks, groups, H, T * picks,
                           dtype_w, lanes_for((H + 7L) / 8)};
    const hipError_t e = by_pair(dtype, dtype_d, [&](auto y, auto d) {
        return launch_k(combine_grad_kernel<decltype(y)::value, decltype(d)::value>, dim3(token_blocks(p.T, p.lanes)), dim3(256),
                        reinterpret_cast<hipStream_t>(stream), p);
    });
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

}  // extern "C"

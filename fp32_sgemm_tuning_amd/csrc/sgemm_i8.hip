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
//   i8_rows_kernel   up to 16 rows of X: bound by W's bytes
//   i8_tile_kernel   tiles through LDS, on the K loop of sgemm_lowp.hpp
//   i8_wide_kernel   many tiles of 256 x 256, on a K loop of their own
//   i8_share_kernel,
//   i8_join_kernel   tiles of a share of K, and the shares added
//   i8_quantize_kernel, i8_dequantize_kernel
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sgemm_rows.hpp"

namespace sgemm_mi355x {

namespace {

using Tile32x32 = TileShape<32, 32, 64, 1, 2, 8, false>;
using Tile64 = TileShape<64, 64, 64, 2, 2, 4, false>;
using Tile128x64 = TileShape<128, 64, 64, 4, 2, 4, false>;
using Tile32x64 = TileShape<32, 64, 64, 1, 4, 4, false>;
using Tile64x128 = TileShape<64, 128, 64, 2, 2, 3, false>;
using TileFourth = TileShape<128, 128, 64, 4, 2, 3, false>;

struct I8Args {
    const char *X, *W;                      // 8-bit integers; rows at multiples of 16 bytes but for i8_rows_kernel<true>
    const float *sx, *sw;
    char *C;
    long ldx, ldw, ldc, strideW, strideS;   // elements; strides from group to group
    const int *offsets;                     // NULL: one group of all rows
    int groups, M, N, K;
    float alpha, beta;
    int dtype_c;
    int *parts;                             // the shares' sums [shares][M][ceil_to(N, 4)]
    int most;                               // tiles of 256 x 256 at most
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

// ---------------------------------------------------------------------------
// Many tiles: 256 x 256, on a K loop of their own.
//
// What a compute unit loads bounds such tiles: 64 KiB per 128 k, for 2048 cycles
// of matrix instructions.  Its first-level cache, 32 KiB of 128-byte lines, also
// holds what is in flight, so a load that takes half of each line it touches (a K
// tile of 64 bytes) leaves half as much in flight and fetches every line twice.
// Here a unit of K is 128 bytes, whole lines of each row (8192 x 14336 x 4096 to
// BF16: 58 -> 29 million reads of the second-level cache, 445 -> 397 us; with all
// that follows 364 to 390 by card and run, mostly 377, 2550 TOPS, of which storing
// 235 MB is about 34).
//
// Five LDS slots of 32 KiB hold the units of A and of B in turn, A_u in slot 2u
// mod 5 and B_u in the next.  Eight waves in two groups, one wave of each on a
// SIMD, read fragments and multiply in turn, half a unit (64 k) at a time, one
// group a phase behind the other; every phase ends with a barrier.  In unit u's
// first read phase the loads of B_{u+1} are issued, in its second those of
// A_{u+2}, into the slots of unit u - 1, which all waves have read by then; the
// wait for unit u + 1 is at the end of the last phase before it is read, and
// leaves A_{u+2} in flight.
//
// A lane holds 16 consecutive columns of a row of C (two pieces of 16 bytes in 16
// bits, see exchange): the rows of B enter the matrix instruction so that its column j of block
// nb is the wave's column 16 * (j / 4) + 4 * nb + j % 4.  A chunk c of row r lies
// at c ^ (r / 2 % 8) in A's slots and at c ^ key_b(r) in B's, whose 16 rows to a
// read differ in bits 0, 1, 4 and 5: no bank conflicts counted in either.
//
// A workgroup per compute unit takes tiles one after another.  The loads of the
// next tile's first units are issued before a tile is stored, and nothing waits
// for the stores until the second unit is read (381 -> 373 us).
struct Wide {
    static constexpr int SLOT = 32768, LDS = 5 * SLOT, NT = 512, WORKGROUPS = 256;
    using Acc = i32x4[8][4];
    struct Tile {
        int g, lo, rows, m0, n0;
        const char *A, *B;                  // the tile's corner in each operand
        int endA, endB;                     // bytes from there to its last row
    };
    const I8Args &p;
    char *lds;
    int lane, wave, units, kr;              // kr: bytes of the remainder unit, which comes first (0: none)
    unsigned to;                            // LDS address of this wave's part of slot 0

    static __device__ __forceinline__ int key_b(int r) { return ((r >> 4) & 3) << 1 | ((r >> 1) & 1); }
    __device__ __forceinline__ Wide(const I8Args &args, char *l) : p(args), lds(l), lane(threadIdx.x & 63) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int K = (p.K + 15) & ~15;
        kr = K % 128;
        if ((p.K & 15) && kr == 0) kr = 128;    // the cut chunk is one of the remainder's
        units = (K - kr) / 128 + (kr != 0);
        to = (unsigned)reinterpret_cast<uintptr_t>((lds_addr_t)lds) + wave * 1024;
    }
    // (in range even if the offsets change while the kernel runs)
    __device__ __forceinline__ void place(Tile &t) const {
        t.A = p.X + min(t.lo + t.m0, p.M - 1) * p.ldx;
        t.B = p.W + t.g * p.strideW + t.n0 * p.ldw;
        t.endA = (min(max(t.rows - t.m0, 1), 256) - 1) * (int)p.ldx;
        t.endB = (min(p.N - t.n0, 256) - 1) * (int)p.ldw;
    }
    // This lane's row of the first 64 of a slot, and the chunk of it that it loads.
    __device__ __forceinline__ int row_of() const { return wave * 8 + (lane >> 3); }
    template <bool B>
    __device__ __forceinline__ int chunk_of() const { return (lane & 7) ^ (B ? key_b(row_of()) : (row_of() >> 1) & 7); }
    // Race-check build: what this lane's loads of a slot fill, before they are issued.
    __device__ __forceinline__ void poison(int slot) const {
        if constexpr (SGEMM_LDS_POISON) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<i32x4 *>(lds + slot * SLOT + wave * 1024 + i * 8192 + 16 * lane) = i32x4{-1, -1, -1, -1};
            wait_lgkmcnt0();
        }
    }
    // `bytes` of each row from `from` on into a slot.  Rows past the operand's last
    // lie behind the descriptor's range, which ends with that row's bytes (a row is
    // as long as the leading dimension at most).
    template <bool B>
    __device__ __forceinline__ void load_rows(const Tile &t, const char *from, int bytes, bool in, int slot) const {
        poison(slot);
        const int ld = (int)(B ? p.ldw : p.ldx);
        const int off = row_of() * ld + 16 * chunk_of<B>();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dma16_lowp(from, (B ? t.endB : t.endA) + bytes, to + slot * SLOT + i * 8192, in ? off + i * 64 * ld : (int)kOutOfRange);
    }
    // Unit u of A or (B) of B into a slot.
    template <bool B>
    __device__ __forceinline__ void load(const Tile &t, int u, int slot) const {
        load_rows<B>(t, (B ? t.B : t.A) + (kr ? u - 1 : u) * 128l, 128, true, slot);
    }
    template <bool B>
    __device__ __forceinline__ void load_first(const Tile &t, int slot) const {
        if (!kr) load<B>(t, 0, slot);
        else load_rows<B>(t, (B ? t.B : t.A) + (((p.K + 15) & ~15) - kr), kr, 16 * chunk_of<B>() < kr, slot);
    }
    // The loads of a tile's first units, into all five slots: no wave reads any.
    __device__ __forceinline__ void begin(const Tile &t) const {
        if (units == 0) return;
        load_first<false>(t, 0);
        load_first<true>(t, 1);
        if (units < 2) return;
        load<false>(t, 1, 2);
        load<true>(t, 1, 3);
        if (units > 2) load<false>(t, 2, 4);
    }
    // acc = the product of a tile that begin() was called for; `landed`: its loads
    // have, and stores may be in flight.  Behind it no wave reads LDS.
    __device__ __forceinline__ void multiply(const Tile &t, Acc &acc, bool landed) const {
#pragma unroll
        for (int mi = 0; mi < 8; ++mi)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) acc[mi][nb] = i32x4{0, 0, 0, 0};
        if (units == 0) return;
        using AL = ALayout<32>;
        const int group = wave >> 2, lr = lane & 15, lg = lane >> 4;
        if (!landed) {                      // unit 0 has landed
            if (units > 2) wait_vm_lgkm0<12>();
            else if (units == 2) wait_vm_lgkm0<8>();
            else wait_vm_lgkm0<0>();
        }
        if (p.K & 15) {                     // what A's rows hold behind K does not count
            if (16 * chunk_of<false>() + 16 == kr) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    i32x4 *chunk = reinterpret_cast<i32x4 *>(lds + wave * 1024 + i * 8192 + 16 * lane);
                    *chunk = first_bytes(*chunk, p.K & 15);
                }
            }
            wait_lgkmcnt0();
        }
        __builtin_amdgcn_s_barrier();
        if (group) __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const int rowb = (wave & 3) * 64 + 16 * (lr >> 2) + (lr & 3);
        // (the second half of a unit: chunks 4 .. 7, bit 6 of the address)
        const int fromA = 4 * AL::offset(group * 128 + lr, lg), fromB = 128 * rowb + 16 * (lg ^ key_b(rowb));
        int sa = 0, u = 0;                  // A_u's slot
        asm volatile("" : "+s"(u));         // (no copy of the loop for its first turn, which would take registers of its own)
        for (; u < units; ++u) {
            const int sb = sa == 4 ? 0 : sa + 1, next = sb == 4 ? 0 : sb + 1, free0 = next == 4 ? 0 : next + 1, free1 = free0 == 4 ? 0 : free0 + 1;
            // the loads of unit u + 1 have landed, those of A_{u+2} may be in flight
            auto next_landed = [&]() {
                if (u == 0 && landed) return;
                if (u + 2 < units) wait_vm_lgkm0<4>();
                else wait_vm_lgkm0<0>();
            };
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const char *A = lds + sa * SLOT + (fromA ^ (64 * ks)), *B = lds + sb * SLOT + (fromB ^ (64 * ks));
                i32x4 fa[8], fb[4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) fb[nb] = *reinterpret_cast<const i32x4 *>(B + nb * 512);
#pragma unroll
                for (int mi = 0; mi < 8; ++mi) fa[mi] = *reinterpret_cast<const i32x4 *>(A + mi * 2048);
                if (ks == 0) {
                    if (u > 0 && u + 1 < units) load<true>(t, u + 1, free0);
                } else {
                    if (u > 0 && u + 2 < units) load<false>(t, u + 2, free1);
                }
                __builtin_amdgcn_sched_barrier(0);
                wait_lgkmcnt0();
                if (ks == 1 && group) next_landed();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int mi = 0; mi < 8; ++mi)
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) acc[mi][nb] = Product<kMulI8>::mfma(fb[nb], fa[mi], acc[mi][nb]);
                __builtin_amdgcn_sched_barrier(0);
                if (ks == 1 && !group) next_landed();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
            sa = next;
        }
        if (!group) __builtin_amdgcn_s_barrier();
    }
    // The scales of a tile's rows (times alpha) and columns, arrived: all loads before them have landed too.
    struct Scales {
        float x[8];
        f32x4 w[4];
    };
    __device__ __forceinline__ void load(const Tile &t, Scales &s) const {
        const int row0 = t.m0 + (wave >> 2) * 128 + (lane & 15), col = t.n0 + (wave & 3) * 64 + 16 * (lane >> 4);
#pragma unroll
        for (int mi = 0; mi < 8; ++mi) s.x[mi] = p.sx[t.lo + max(min(row0 + mi * 16, t.rows - 1), 0)];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) s.w[nb] = scales4(p.sw + t.g * p.strideS, col + 4 * nb, p.N);
#pragma unroll
        for (int mi = 0; mi < 8; ++mi) {
            s.x[mi] *= p.alpha;
            asm volatile("" : "+v"(s.x[mi]));
        }
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) asm volatile("" : "+v"(s.w[nb]));
    }
    // C of a tile.
    __device__ __forceinline__ void store(const Tile &t, const Acc &acc, const Scales &s) const {
        int l = threadIdx.x & 63;
        asm volatile("" : "+v"(l));         // (what follows from it is not kept in registers from tile to tile)
        const bool low = (l & 15) < 8;
        const int row0 = t.m0 + (wave >> 2) * 128, n0 = t.n0 + (wave & 3) * 64, col = n0 + 16 * (l >> 4);
        by_result(p.dtype_c, [&](auto f16, auto out16) {
            constexpr bool F16 = decltype(f16)::value, OUT16 = decltype(out16)::value;
            auto value = [&](int mi, int nb) { return to_float(acc[mi][nb]) * s.x[mi] * s.w[nb]; };
            auto at = [&](int row) { return p.C + (t.lo + (long)row) * p.ldc * (OUT16 ? 2 : 4); };
            if (OUT16 && p.beta == 0.f && t.n0 + 256 <= p.N) {
                i32x4 o[8][2];              // all values, then all stores
#pragma unroll
                for (int mi = 0; mi < 8; ++mi) {
                    __builtin_amdgcn_sched_barrier(0);  // (eight rows at once need more registers than there are)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const i32x2 x = round16<F16>(value(mi, 2 * h)), y = round16<F16>(value(mi, 2 * h + 1));
                        o[mi][h] = i32x4{x[0], x[1], y[0], y[1]};
                    }
                }
                wait_vmcnt0();
#pragma unroll
                for (int mi = 0; mi < 8; ++mi) {
                    exchange(o[mi][0], o[mi][1], low);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = row0 + mi * 16 + 8 * h + (l & 7);
                        if (row < t.rows) __builtin_memcpy(at(row) + 2l * (col + (low ? 0 : 8)), &o[mi][h], 16);
                    }
                }
                return;
            }
            wait_vmcnt0();
#pragma unroll
            for (int mi = 0; mi < 8; ++mi) {
                __builtin_amdgcn_sched_barrier(0);
                f32x4 v[4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) v[nb] = value(mi, nb);
                if constexpr (OUT16) {
                    const int row = row0 + mi * 16 + (l & 15);
                    if (row >= t.rows) continue;
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) store4<F16, OUT16>(at(row), col + 4 * nb, p.N, p.beta, v[nb]);
                } else {
                    turn(v);
#pragma unroll
                    for (int i = 0; i < 4; i += 2) exchange(v[i], v[i + 1], low);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = row0 + mi * 16 + 8 * (i & 1) + (l & 7);
                        if (row >= t.rows) continue;
                        const int c = n0 + 4 * (l >> 4) + 16 * (i & ~1) + (low ? 0 : 16);
                        store4<F16, OUT16>(at(row), c, p.N, p.beta, v[i]);
                    }
                }
            }
        });
    }
    // The lanes of rows r (low) and r + 8 hold the pieces a and b of theirs: a becomes row r's and b row r + 8's,
    // the first piece in the low lane and the second in the other.  A wave's store then writes whole lines of
    // 128 bytes of eight rows, not halves of sixteen (8192 x 8192 x 2048 in 136 -> 132.5 us, 4096^3 in 60 -> 57.5).
    template <class V> static __device__ __forceinline__ void exchange(V &a, V &b, bool low) {
        i32x4 x = __builtin_bit_cast(i32x4, a), y = __builtin_bit_cast(i32x4, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int other = __builtin_amdgcn_mov_dpp(low ? y[i] : x[i], 0x128, 0xf, 0xf, true);   // (8 lanes on)
            const int first = low ? x[i] : other, second = low ? other : y[i];
            x[i] = first;
            y[i] = second;
        }
        a = __builtin_bit_cast(V, x);
        b = __builtin_bit_cast(V, y);
    }
    // Lane group l/16 = j gets of lane group i (block j) as its block i.
    static __device__ __forceinline__ void turn(f32x4 (&v)[4]) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            unsigned x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __float_as_uint(v[i][r]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto y = __builtin_amdgcn_permlane32_swap(x[i], x[i + 2], false, false);
                x[i] = y[0];
                x[i + 2] = y[1];
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const auto y = __builtin_amdgcn_permlane16_swap(x[i], x[i + 1], false, false);
                x[i] = y[0];
                x[i + 1] = y[1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i][r] = __uint_as_float(x[i]);
        }
    }
};

// Tiles of 256 x 256, in rounds of one per compute unit; the tiles of a last round
// that fills at most half of the chip are cut in two or four, a part for each
// workgroup, as in Mixed.  One workgroup per compute unit does it all: more would
// wait for LDS and cost 3 us at the end.
template <class T>
__device__ __forceinline__ void i8_part(const TileList<256, I8Args> &list, char *lds, int id, int sub) {
    int g = 0, lo = 0, rows = 0, tm = 0, tn = 0, m0, n0;
    list.find(id, g, lo, rows, tm, tn);
    part_corner<T>(tm, tn, sub, m0, n0);
    if (m0 < rows && n0 < list.p.N) i8_tile<T>(list.p, lds, g, lo, rows, m0, n0);
}

__global__ void __launch_bounds__(Wide::NT) i8_wide_kernel(I8Args p) {
    __shared__ __attribute__((aligned(16))) char lds[Wide::LDS];
    constexpr int W = Wide::WORKGROUPS;
    const TileList<256, I8Args> list(p, 256, p.most);
    const int whole = list.total & ~(W - 1), rest = list.total - whole, upto = rest > W / 2 ? list.total : whole;
    int id = blockIdx.x;
    if (id < upto) {
        const Wide wide(p, lds);
        Wide::Tile t = {};
        auto find = [&](int n) {
            int tm = 0, tn = 0;
            list.find(n < whole ? xcd_run(n, whole) : whole + xcd_run(n - whole, rest), t.g, t.lo, t.rows, tm, tn);
            t.m0 = tm * 256;
            t.n0 = tn * 256;
            wide.place(t);
        };
        Wide::Acc acc;
        find(id);
        wide.begin(t);
        for (bool landed = false;; landed = true) {
            wide.multiply(t, acc, landed);
            const Wide::Tile done = t;
            id += W;
            if (id < upto) {
                find(id);
                wide.begin(t);
            }
            Wide::Scales s;
            wide.load(done, s);
            wide.store(done, acc, s);
            if (id >= upto) break;
        }
    }
    if (upto == list.total) return;
    const int k = blockIdx.x;
    if (rest > W / 4) {
        if (k >= 2 * rest) return;
        const int at = xcd_run(k, 2 * rest);
        i8_part<TileTall>(list, lds, whole + (at >> 1), at & 1);
    } else if (k < 4 * rest) {
        const int at = xcd_run(k, 4 * rest);
        i8_part<TileFourth>(list, lds, whole + (at >> 2), at & 3);
    }
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

// One lane's 16 integers of a row from k on, of which `left` are left: those from
// there on 0 (CUT), or whatever lies in an aligned chunk.
template <bool ANY, bool CUT>
__device__ __forceinline__ i32x4 row_chunk(const char *at, int left) {
    i32x4 v = {0, 0, 0, 0};
    if constexpr (!ANY) {
        if (left > 0) v = *reinterpret_cast<const i32x4 *>(at);
        return CUT && left < 16 ? first_bytes(v, left) : v;
    }
    if (left >= 16) {                       // from whole words: those at odd bytes load far slower
        const unsigned past = reinterpret_cast<uintptr_t>(at) & 3;
        const int *word = reinterpret_cast<const int *>(at - past);
        __builtin_memcpy(&v, word, 16);
        const int fifth = word[past ? 4 : 3];                   // (holds the 16th byte, or is one that was loaded)
        const i32x4 up = {v[1], v[2], v[3], fifth};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (int)__builtin_amdgcn_alignbyte((unsigned)up[i], (unsigned)v[i], past);
        return v;
    }
    for (int e = 0; e < left; ++e) v[e >> 2] |= (int)((unsigned)(unsigned char)at[e] << (8 * (e & 3)));
    return v;
}

// Up to 16 rows and few columns: a block of 16 rows of W per workgroup, whose eight
// waves take shares of K of their own, so that no wave waits for another's loads
// and nothing passes through LDS but the sums at the end.  A lane's 16 bytes of a
// row are its operand of one v_mfma_i32_16x16x64_i8 as they lie in memory; two
// steps read a row's 128-byte line, and four lines of every row are in flight.
// 1 x 4096 x 4096: 6.3 us, where tiles of 32 x 32 take 8.1; from two blocks per
// compute unit on those are faster for many rows (16 x 8192 x 4096: 13.1 and 10.5; not
// for one, 9.3 and 10.3; 1 x 14336 x 4096: 15.0 and 15.7).  ANY: rows of any
// alignment, which the tiles would have to copy first (8 x 4096 x 4095 18.1 -> 12.8
// us, 16 x 14336 x 4095 41.4 -> 40.2), slower all the same than aligned ones (8.7 and
// 15.9): two loads for 16 bytes.
template <bool ANY>
__global__ void __launch_bounds__(512) i8_rows_kernel(I8Args p) {
    constexpr int NW = 8, AHEAD = 4;
    __shared__ i32x4 part[NW][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4, n0 = blockIdx.x * 16;
    // (rows past the last: that one again, for outputs that are not stored)
    const char *x = p.X + min(lr, p.M - 1) * p.ldx + 16 * lg, *w = p.W + min(n0 + lr, p.N - 1) * p.ldw + 16 * lg;
    i32x4 acc = {0, 0, 0, 0};
    const int lines = (p.K + 127) / 128, last = lines * (wave + 1) / NW;
    for (int c0 = lines * wave / NW; c0 < last; c0 += AHEAD) {
        i32x4 fx[AHEAD][2], fw[AHEAD][2];
        const bool whole = min(c0 + AHEAD, last) * 128 <= p.K;
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
            if (c0 + t >= last) break;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = (c0 + t) * 128 + 64 * s, left = whole ? 16 : p.K - k - 16 * lg;    // integers from this lane's chunk on
                if (whole) {
                    fw[t][s] = row_chunk<ANY, false>(w + k, 16);
                    fx[t][s] = row_chunk<ANY, false>(x + k, 16);
                } else {
                    fw[t][s] = row_chunk<ANY, false>(w + k, left);
                    fx[t][s] = row_chunk<ANY, true>(x + k, left);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
            if (c0 + t >= last) break;
#pragma unroll
            for (int s = 0; s < 2; ++s) acc = Product<kMulI8>::mfma(fw[t][s], fx[t][s], acc);
        }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 1; i < NW; ++i) acc += part[i][lane];
    const int col = n0 + 4 * lg;            // columns .. +3 of row lr
    if (lr >= p.M || col >= p.N) return;
    const f32x4 c = to_float(acc) * (p.alpha * p.sx[lr]) * scales4(p.sw, col, p.N);
    by_result(p.dtype_c, [&](auto f16, auto out16) {
        store4<decltype(f16)::value, decltype(out16)::value>(p.C + lr * p.ldc * (decltype(out16)::value ? 2 : 4), col, p.N, p.beta, c);
    });
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
// below 2^24 of them), is doubled and compared with a step.  (Not halved steps:
// half of an odd multiple of 2^-149, which an s below 2^-125 can be, is no FP32
// value.)
__device__ __forceinline__ int nearest(float x, float s, float inverse) {
    const float y = x * inverse;
    float q = rintf(y);
    if (fabsf(fabsf(y - q) - 0.5f) < 0x1p-12f) {
        const float rest = __builtin_fmaf(-q, s, x), twice = 2.f * fabsf(rest);
        if (twice > s || (twice == s && ((int)q & 1))) q += rest > 0.f ? 1.f : -1.f;
    }
    return (int)q;
}

// A row per NT threads, 8 values to a thread and step, PIECES steps of them in
// registers; longer rows are read again (from the cache).  The largest
// magnitude is taken as bits: NaN lies above infinity there, and either makes
// the scale NaN.  16384 x 4096 in BF16: 45 to 48 us, 4.3 TB/s (four steps in
// registers, which short rows leave empty, 52); back 34 us, 5.8 TB/s.
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
    for (int d = NT < 64 ? NT / 2 : 32; d; d >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, d));
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

// The forms of one weight's product.  Each but the first is priced as
//   3.5 us + rounds over the compute units * K / 128 * its time for 128 k of a tile,
// and the cheapest taken.  Those times lie at or between those of weights that stay
// in the caches and those of weights that come from memory.  At K = 4096, BF16
// results, in us: priced (measured from the caches, from memory)
//   32 x 32      64 x 4096   7.8 (7.4, 10.2)     two at once   64 x 8192  10.2 (9.9, 14.8)
//   64 x 64     200 x 4096  10.5 (9.8, 13.8)     two at once  256 x 8192  22.1 (16.8, 23.0)
//   128 x 64    512 x 4096  17.3 (14.9, 19.4)
//   256 x 256, whole rounds: 4096 x 4096  56.3 (56.8, 61.8);
//   in halves 1024 x 8192   39.7 (38.6, 39.9);   in quarters 1024 x 4096  22.7 (22.4, 25.5)
// From memory the form taken is the fastest within 3% at 64 to 1024 rows of 4096 x
// 4096, 8192 x 4096 and 2048 x 8192; not at 1 x 8192 x 4096 (32 x 32: 10.3, the rows'
// kernel 9.3) and 100 x 1000 x 8192 (eight shares 12.6, 32 x 32 11.8).  A grid of 64 x
// 64 tiles that leaves most of the chip idle splits K: 100 x 1000 x 8192 14.7 -> 9.8
// from the caches, 21.1 -> 12.6 from memory.
enum Form { kRows, kTile32, kTile64, kTile128x64, kWide };

struct Plan {
    Form form;
    int shares;
};

// `copies`: whether an operand would be copied for all forms but kRows.
Plan select_plan(int M, int N, int K, bool copies) {
    auto tiles = [&](int bm, int bn) { return (M + bm - 1L) / bm * ((N + bn - 1L) / bn); };
    const double steps = std::max(1, (K + 127) / 128);
    if (M <= 16 && (N <= 16 * 256 || (copies && launch_fits((N + 15L) / 16, 512)))) return {kRows, 1};
    Plan best = {kTile32, 1};
    double least = 1e30;
    auto offer = [&](Form form, int shares, double us) {
        if (us < least) least = us, best = {form, shares};
    };
    auto paired = [](double load, double one, double two) {
        const double full = std::floor(load / 512), rest = load - 512 * full;
        return full * two + (rest > 256 ? two : rest > 0 ? one : 0);
    };
    const long t64 = tiles(64, 64), t256 = tiles(256, 256);
    offer(kTile32, 1, 3.5 + steps * paired(tiles(32, 32), 0.134, 0.21));
    offer(kTile64, 1, 3.5 + steps * paired(t64, 0.22, 0.58));
    for (int s = 2; s <= 8 && t64 * s <= 256; s *= 2)
        offer(kTile64, s, 6.5 + std::ceil(steps / s) * 0.22 + s * 8e-6 * M * N / 3.5);
    offer(kTile128x64, 1, 3.5 + steps * 0.43 * std::ceil(tiles(128, 64) / 256.0));
    const double whole = std::floor(t256 / 256.0), rest = t256 - 256 * whole;
    offer(kWide, 1, 3.5 + steps * (1.65 * (whole + (rest > 128)) + (rest > 128 || rest == 0 ? 0 : rest > 64 ? 1.13 : 0.6)));
    return best;
}

template <class T>
hipError_t launch_tiles(const I8Args &p, hipStream_t s) {
    return launch_k(i8_tile_kernel<T>, dim3((unsigned)most_tiles(p.groups, p.M, p.N, T::BM, T::BN)), dim3(T::NT), s, p);
}

template <class T>
hipError_t launch_shares(const I8Args &p, int shares, hipStream_t s) {
    const hipError_t e = launch_k(i8_share_kernel<T>, dim3((unsigned)most_tiles(1, p.M, p.N, T::BM, T::BN), (unsigned)shares), dim3(T::NT), s, p);
    if (e != hipSuccess) return e;
    return launch_k(i8_join_kernel, dim3((unsigned)(((p.N + 3L) / 4 * p.M + 255) / 256)), dim3(256), s, p, shares);
}

hipError_t launch_wide(I8Args p, hipStream_t s) {
    p.most = (int)most_tiles(p.groups, p.M, p.N, 256, 256);
    return launch_k(i8_wide_kernel, dim3(Wide::WORKGROUPS), dim3(Wide::NT), s, p);
}

// (what the counts of tiles stay below)
bool wide_fits(int groups, int M, int N) { return launch_fits(most_tiles(groups, M, N, 256, 256), Wide::NT); }

hipError_t launch_dense(const I8Args &p, Plan plan, bool copies, hipStream_t s) {
    switch (plan.form) {
        case kRows: return launch_k(copies ? i8_rows_kernel<true> : i8_rows_kernel<false>, dim3((unsigned)((p.N + 15) / 16)), dim3(512), s, p);
        case kTile32: return launch_tiles<Tile32x32>(p, s);
        case kTile64: return plan.shares > 1 ? launch_shares<Tile64>(p, plan.shares, s) : launch_tiles<Tile64>(p, s);
        case kTile128x64: return launch_tiles<Tile128x64>(p, s);
        default: return launch_wide(p, s);
    }
}

// Whether one launch can cover the outputs.
bool dense_fits(Plan plan, int M, int N) {
    switch (plan.form) {
        case kRows: return true;
        case kTile32: return launch_fits(most_tiles(1, M, N, 32, 32), Tile32x32::NT);
        case kTile64: return launch_fits(most_tiles(1, M, N, 64, 64), Tile64::NT);
        case kTile128x64: return launch_fits(most_tiles(1, M, N, 128, 64), Tile128x64::NT);
        default: return wide_fits(1, M, N);
    }
}

// By the rows of an average group.  In us, 16 groups of 2048 x 4096 with weights from
// memory:
//   rows     128    512   1024   1536   2048   2560   4096
//   32 x 64   33.4   37.2  47.9   55.3   65.2   76.5  108
//   64 x 128  35.6   37.2  41.2   41.7   53.2   55.3   75.4
//   256 x 256 36.1   38.5  40.1   42.0   43.7   45.8   58.9
// (2048 rows: groups of 112 to 148, for which the rule takes 64 x 128.)  Few groups, or
// few columns, leave most of the chip idle, which the rule does not look at: 520 rows in
// 2 groups of 1024 x 4096 18.4 on 256 x 256, 10.8 on 64 x 64; 200 rows by one weight of
// 64 x 4096 17.1 and 10.4, on 32 x 64 9.1.
hipError_t launch_grouped(const I8Args &p, hipStream_t s) {
    const int rows = p.M / std::min(p.groups, p.M);
    return rows <= 32 ? launch_tiles<Tile32x64>(p, s) : rows <= 128 ? launch_tiles<Tile64x128>(p, s) : launch_wide(p, s);
}

bool grouped_fits(int groups, int M, int N) {
    const int rows = groups > 0 && M > 0 ? M / std::min(groups, M) : 0;
    return rows <= 32    ? launch_fits(most_tiles(groups, M, N, 32, 64), Tile32x64::NT)
           : rows <= 128 ? launch_fits(most_tiles(groups, M, N, 64, 128), Tile64x128::NT)
                         : wide_fits(groups, M, N);
}

constexpr int kMaxK8 = (1 << 17) - 1;       // sums of products of -128 fit 32 bits
constexpr long kMaxLd8 = 2L * kMaxLd16;
constexpr int kMaxGroups8 = 65534;          // launch grid extent of the padded copies, X's among them

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

Needs dense_needs(Plan plan, int M, int N, int K, const void *X, int ldx, const void *W, int ldw) {
    return plan.form == kRows ? Needs{0, 0, 0} : i8_needs(1, M, N, K, X, ldx, W, ldw, 0, plan.shares);
}

// Rows of any alignment into rows of whole aligned chunks, zeros behind them.
struct PadJob {
    const char *src;
    char *dst;
    long ld, stride;                        // bytes; from matrix to matrix
    int rows;                               // of each matrix
};

// Matrix 0 of blockIdx.y is X, the others W's (or all W's: first 0).  A row per
// wave and turn, a 16-byte chunk per lane.
__global__ void __launch_bounds__(256) pad_bytes_kernel(PadJob x, PadJob w, int first, int K) {
    const bool is_w = (int)blockIdx.y >= first;
    const PadJob &j = is_w ? w : x;
    const long at = is_w ? blockIdx.y - first : 0, ld = ((long)K + 15) & ~15l;
    const char *src = j.src + at * j.stride;
    char *dst = j.dst + at * j.rows * ld;
    for (long r = blockIdx.x * 4l + (threadIdx.x >> 6); r < j.rows; r += gridDim.x * 4l) {
        const char *from = src + r * j.ld;
        for (int c = 16 * (threadIdx.x & 63); c < K; c += 1024) {
            i32x4 v = {0, 0, 0, 0};
            if (c + 16 <= K) {
                __builtin_memcpy(&v, from + c, 16);     // (bound by memory; whole words and a shift are no faster here)
            } else {
                for (int e = 0; c + e < K; ++e) v[e >> 2] |= (int)((unsigned)(unsigned char)from[c + e] << (8 * (e & 3)));
            }
            *reinterpret_cast<i32x4 *>(dst + r * ld + c) = v;
        }
    }
}

// The copies that the operands need, made in the workspace by one launch.
hipError_t take_operands(I8Args &p, const Needs &need, char *w, hipStream_t s) {
    p.parts = reinterpret_cast<int *>(w + need.x + need.w);
    if (need.x + need.w == 0) return hipSuccess;
    const PadJob jx = {p.X, w, p.ldx, 0, p.M}, jw = {p.W, w + need.x, p.ldw, p.strideW, p.N};
    const int first = need.x ? 1 : 0, rows = std::max(need.x ? p.M : 0, need.w ? p.N : 0);
    const hipError_t e = launch_k(pad_bytes_kernel, dim3((unsigned)std::min((rows + 3L) / 4, 1L << 20), (unsigned)(first + (need.w ? p.groups : 0))),
                                  dim3(256), s, jx, jw, first, p.K);
    if (need.x) {
        p.X = w;
        p.ldx = ceil_to(p.K, 16);
    }
    if (need.w) {
        p.W = w + need.x;
        p.ldw = ceil_to(p.K, 16);
        p.strideW = p.N * p.ldw;
    }
    return e;
}

bool workspace_ok(long need, const void *workspace, long long bytes) {
    return need == 0 || (workspace != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(workspace) & 15) == 0);
}

constexpr int kShortRow = 256, kWaveRow = 1024;    // longest rows that 16 lanes and a wave quantise (in registers; a workgroup holds 4096)
constexpr int kMaxRows8 = 1 << 24;          // launch grid extents
constexpr int kMaxRowQ = 1 << 30;           // (a row's last step stays in 32 bits)

int check_quant(int dtype, int M, int K, int ldv, int ldx) {
    if (!dtype_ok(dtype)) return SGEMM_STATUS_INVALID_DTYPE;
    return M < 0 || K < 0 || K > kMaxRowQ || ldx < std::max(K, 1) || ldv < std::max(K, 1) ? SGEMM_STATUS_INVALID_DIM : SGEMM_STATUS_OK;
}

}  // namespace
}  // namespace sgemm_mi355x

using namespace sgemm_mi355x;

extern "C" {

long long sgemm_i8_workspace(int M, int N, int K, const void *X, int ldx, const void *W, int ldw) {
    if (M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_DIM;
    return dense_needs(select_plan(M, N, K, !chunk_rows8(X, ldx) || !chunk_rows8(W, ldw)), M, N, K, X, ldx, W, ldw).all();
}

int sgemm_i8(int M, int N, int K, float alpha, const void *X, int ldx, const float *x_scales, const void *W, int ldw,
             const float *w_scales, float beta, void *C, int ldc, int dtype_c, void *workspace, long long workspace_bytes,
             void *stream) {
    if (!dtype_ok(dtype_c)) return SGEMM_STATUS_INVALID_DTYPE;
    if (M < 0 || M > kMaxRows8 || N < 0 || N > (1 << 30) || K < 0 || K > kMaxK8) return SGEMM_STATUS_INVALID_DIM;
    if (ldx < std::max(K, 1) || ldw < std::max(K, 1) || ldc < std::max(N, 1)) return SGEMM_STATUS_INVALID_DIM;
    const bool copies = !chunk_rows8(X, ldx) || !chunk_rows8(W, ldw);
    const Plan plan = select_plan(M, N, K, copies);
    if (!dense_fits(plan, M, N)) return SGEMM_STATUS_INVALID_DIM;
    if (M == 0 || N == 0) return SGEMM_STATUS_OK;
    if (C == nullptr || x_scales == nullptr || w_scales == nullptr || (K > 0 && (X == nullptr || W == nullptr)))
        return SGEMM_STATUS_NULL_POINTER;
    const Needs need = dense_needs(plan, M, N, K, X, ldx, W, ldw);
    if (!workspace_ok(need.all(), workspace, workspace_bytes)) return SGEMM_STATUS_SCRATCH_TOO_SMALL;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    I8Args p = {static_cast<const char *>(X), static_cast<const char *>(W), x_scales, w_scales, static_cast<char *>(C),
                ldx, ldw, ldc, 0, 0, nullptr, 1, M, N, K, alpha, beta, dtype_c, nullptr, 0};
    hipError_t e = take_operands(p, need, static_cast<char *>(workspace), s);
    if (e == hipSuccess) e = launch_dense(p, plan, copies, s);
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
                ldx, ldw, ldc, stride_w, stride_s, offsets, groups, M, N, K, alpha, beta, dtype_c, nullptr, 0};
    hipError_t e = take_operands(p, need, static_cast<char *>(workspace), s);
    if (e == hipSuccess) e = launch_grouped(p, s);
    return e == hipSuccess ? SGEMM_STATUS_OK : hip_status(e, "kernel launch");
}

int sgemm_i8_quantize(int dtype, int M, int K, const void *X, int ldx, void *values, int ldv, float *scales, void *stream) {
    const int st = check_quant(dtype, M, K, ldv, ldx);
    if (st != SGEMM_STATUS_OK) return st;
    if (!launch_fits(K <= kShortRow ? (M + 15L) / 16 : K <= kWaveRow ? (M + 3L) / 4 : M, 256)) return SGEMM_STATUS_INVALID_DIM;
    if (M == 0) return SGEMM_STATUS_OK;
    if (scales == nullptr || (K > 0 && (X == nullptr || values == nullptr))) return SGEMM_STATUS_NULL_POINTER;
    const QuantArgs p = {static_cast<const char *>(X), static_cast<signed char *>(values), scales, nullptr, ldx, ldv, M, K};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = by_dtype(dtype, [&](auto d) {
        constexpr int D = decltype(d)::value;
        return p.K <= kShortRow ? launch_k(i8_quantize_kernel<D, 16>, dim3((unsigned)((p.M + 15L) / 16)), dim3(256), s, p)
               : p.K <= kWaveRow ? launch_k(i8_quantize_kernel<D, 64>, dim3((unsigned)((p.M + 3L) / 4)), dim3(256), s, p)
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

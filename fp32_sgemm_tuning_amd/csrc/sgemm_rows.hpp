// Tiles of products whose rows come in groups, the groups' bounds known to the
// device only: how a workgroup finds its tile.
#pragma once

#include <algorithm>

#include "sgemm_tile16.hpp"

namespace sgemm_mi355x {

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

// The groups' tiles of BM rows one after another (of arguments P with groups, M, N
// and rows_of(g, lo, rows)): how many there are, at most
// `most`, and the group and the tile of number `id`.  Wave-uniform.  (Groups that
// overlap, in offsets that decrease, can have more tiles than the grid covers and
// than 32 bits count: products with the number of tile columns are formed in 64.
// The tile rows of 64 groups fit 32 bits: 64 * 2^31 / 256, and M is at most 65535
// times 32 or 128 where BM is less.)
template <int BM, class P>
struct TileList {
    const P &p;
    int tiles_n, first, total;                  // first: tile rows of group `lane`
    __device__ __forceinline__ int tile_rows(int g) const {
        int l = 0, r = 0;
        if (g < p.groups) p.rows_of(g, l, r);
        return (r + BM - 1) / BM;
    }
    __device__ __forceinline__ TileList(const P &args, int bn, int most) : p(args), tiles_n((args.N + bn - 1) / bn) {
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
                p.rows_of(base + at, lo, rows);
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

// The most tiles of bm x bn that any split of the rows into groups can have.
inline long most_tiles(int groups, int M, int N, int bm, int bn) {
    const long most = std::min(groups, M);
    return (M + most * (bm - 1)) / bm * ((N + bn - 1) / bn);
}

}  // namespace sgemm_mi355x

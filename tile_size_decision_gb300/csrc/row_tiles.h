// The lookup of a row tile among ragged groups, by one warp.  Free of CUDA's
// types and intrinsics: `Warp` supplies lane(), ballot(), first() (index of the
// lowest set bit), shfl() and shfl_up(), so that a host program can run the
// same lookup on 32 threads.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TILES_WARP_FN __device__ __forceinline__
#else
#define TILES_WARP_FN inline
#endif

namespace tiles {

// Rows [row0, end) of one tile of `group`.
struct RowTile { int group, row0, end; };

TILES_WARP_FN int clamp_offset(int v, int m) { return v < 0 ? 0 : v > m ? m : v; }

// Tile `want` among the groups' tiles of `tile_rows` rows, in group order; a
// warp looks at 32 groups at a time and keeps the 32 that it is at, so that the
// next lookup among the same ones costs a vote and shuffles.  Any order of
// `want` is right, an ascending one is quick: a tile before the groups at hand
// starts over at the first.
template <typename Warp>
struct RowTileLookup {
    int base = 0, g0 = -32;           // tiles before the chunk; its first group
    int lo = 0, hi = 0, upto = 0, tiles = 0, total = 0;

    // False past the last tile.
    TILES_WARP_FN bool seek(const int32_t* offsets, int groups, int m, int tile_rows, int want,
                            RowTile* out) {
        const int lane = Warp::lane();
        if (want < base) { base = total = 0; g0 = -32; }
        while (want >= base + total) {
            if (g0 + 32 >= groups) return false;
            g0 += 32;
            base += total;
            const int g = g0 + lane;
            lo = hi = 0;
            if (g < groups) {
                lo = clamp_offset(offsets[g], m);
                hi = clamp_offset(offsets[g + 1], m);
            }
            tiles = hi > lo ? (hi - lo + tile_rows - 1) / tile_rows : 0;
            upto = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int t = Warp::shfl_up(upto, d);
                if (lane >= d) upto += t;
            }
            total = Warp::shfl(upto, 31);
        }
        const int src = Warp::first(Warp::ballot(want < base + upto));
        const int first = base + Warp::shfl(upto - tiles, src);
        out->group = g0 + src;
        out->row0 = Warp::shfl(lo, src) + (want - first) * tile_rows;
        out->end = Warp::shfl(hi, src);
        return true;
    }
};

}  // namespace tiles

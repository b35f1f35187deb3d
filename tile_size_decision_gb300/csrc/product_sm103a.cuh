// What the product kernels (dense 8-bit, grouped 16- and 8-bit, and the
// grouped weight gradient) share: their arguments, the lookup of a tile among
// ragged groups, and their host-side launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm_sm103a.cuh"
#include "launch_util.h"
#include "op_ptx.cuh"
#include "row_tiles.h"

namespace tiles {

constexpr int kScaleBlock = 128;      // columns (and weight rows) per scale
constexpr int kMaxGroups = 4096;

// Operand kinds of the products.
constexpr int kWeight16KN = 0;        // 16-bit, b is k x n (MN-major weight)
constexpr int kWeight16NK = 1;        // 16-bit, b is n x k (K-major weight)
constexpr int kWeight8NK = 2;         // e4m3, b is n x k, block scales
constexpr int kWeightGrad = 3;        // 16-bit weight gradient (the large-tile kernel's form)

struct ProductArgs {
    int32_t m, n, k;
    int32_t groups;                   // 0: dense
    const int32_t* offsets;
    int32_t n_blocks, k_blocks;       // of the kernel's tile
    int32_t split;                    // few rows: CTAs along K (a cluster)
    int32_t tile_cols;                // 8-bit pairs: weight rows a tile, a multiple of 32
    int32_t tma_store;                // pairs: c leaves through TMA stores (its map is valid)
    int64_t stride_c;                 // weight gradient: elements between groups' results
    void* c;
    int64_t ldc;
    int32_t c_dtype;
    uint32_t idesc;
    const float* sa;
    const float* sb;
    int64_t sa_row, sa_block, sb_row, sb_block, sb_group;
    int32_t* err;
    uint64_t wait_limit_ns;
    int32_t drop_stage;               // test hook (-1: none)
};

// How long a wait of the large-tile kernels may take.  Once one has expired in
// this call, the CTAs that start later, which may miss the same thing, give up
// soon: a call of many units then ends too, in seconds.
__device__ __forceinline__ uint64_t wait_limit(const ProductArgs& a) {
    const uint64_t after = 10000000ull;
    return *static_cast<const volatile int32_t*>(a.err) != 0 && a.wait_limit_ns > after
               ? after : a.wait_limit_ns;
}

// The lanes of a warp, as the lookup of a row tile uses them.
struct WarpLanes {
    static __device__ __forceinline__ int lane() { return threadIdx.x & 31; }
    static __device__ __forceinline__ unsigned ballot(bool p) { return __ballot_sync(0xffffffffu, p); }
    static __device__ __forceinline__ int first(unsigned mask) { return __ffs(mask) - 1; }
    static __device__ __forceinline__ int shfl(int v, int src) { return __shfl_sync(0xffffffffu, v, src); }
    static __device__ __forceinline__ int shfl_up(int v, int d) { return __shfl_up_sync(0xffffffffu, v, d); }
};

// A pair's units come from cluster launch control, which promises a cluster
// that has not started and no order among them.
using RowTileCursor = RowTileLookup<WarpLanes>;

// One value in the output's type.
__device__ __forceinline__ void store_one(void* c, int64_t at, float v, int dtype) {
    if (dtype == TILES_F32) static_cast<float*>(c)[at] = v;
    else if (dtype == TILES_F16) static_cast<__half*>(c)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(c)[at] = __float2bfloat16_rn(v);
}

// The few-rows kernel: tile_rows in {16, 32, 64}; units is the number
// of (row tile, weight block) pairs launched.
int launch_stream(int kind, int tile_rows, const CUtensorMap& weight, const CUtensorMap& rows,
                  const ProductArgs& args, int64_t units, cudaStream_t st);

// The 16-bit kernel on CTA pairs: tiles of 256 weight columns by up to 256
// rows (weight gradient: dc's columns by a's); units is an upper bound.  rows
// has boxes of 32 rows, rows128 of 128 (weight gradient: not used).
int launch_pair(int kind, const CUtensorMap& weight, const CUtensorMap& rows,
                const CUtensorMap& rows128, const CUtensorMap& out, const ProductArgs& args,
                int units, cudaStream_t st);
// The 8-bit kernel on CTA pairs: tiles of 256 rows by args.tile_cols weight
// rows; units is an upper bound.
int launch_pair8(const CUtensorMap& weight, const CUtensorMap& rows, const CUtensorMap& out,
                 const ProductArgs& args, int units, cudaStream_t st);
// CTA pairs resident at once on the current device.
int pair_max_groups(int sms);

}  // namespace tiles

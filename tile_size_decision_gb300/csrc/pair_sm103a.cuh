// What the two kernels on CTA pairs share (16-bit products and gradients, and
// 8-bit products): the stage geometry, the barriers and the walk through the
// grid's units.
#pragma once

#include "product_sm103a.cuh"

namespace tiles {
namespace {

constexpr int kThreads = 384;
constexpr int kStages = 6;
constexpr int kHalfBytes = 128 * 128;                 // one operand of a stage, per CTA
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kAtomBytes = 64 * 128;
constexpr int kBoxRows = 32;                          // rows per TMA box of the MMA's N operand
constexpr int kMaxWidth = 256;                        // TMEM columns of a tile
// Epilogue staging, per warp: 32 rows of 64 bytes, padded so that eight
// 16-byte accesses to successive rows hit distinct banks.
constexpr int kStagePitch = 80;
constexpr int kStagingBytes = 8 * 32 * kStagePitch;
constexpr int kBarrierBytes = 768;

struct PairBarriers {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
    uint64_t side_full[8], side_empty[8];             // scales (8-bit), ragged ends (gradient)
    uint64_t drain;
    uint64_t next_full[2], next_empty[2];
    ulonglong2 next[2];                               // answers about the next unit
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(PairBarriers) <= kBarrierBytes, "barrier block too large");

// The pair's units in turn: its own, then those of clusters that have not
// started yet, which the leader's TMA warp claims a unit ahead.  Every role's
// warp walks through the same answers.  (The units are uneven where groups
// are: a fixed assignment left pairs idle for a fifth of the time on the
// weight gradient of 16 uneven groups.)
struct Walk {
    int unit;
    uint32_t slot = 0, phase = 0;

    // The answer for the unit after this one; false at the end (or on an
    // expired wait, *failed).
    __device__ __forceinline__ bool next(PairBarriers* bar, const volatile int* abort,
                                         uint64_t limit, bool* failed) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->next_full[slot], phase, abort, limit))) {
            *failed = true;
            return false;
        }
        const int x = ptx::cancelled_cta_x(&bar->next[slot]);
        // Read before the next answer is written here (by the async proxy).
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            ptx::mbar_arrive_remote(ptx::map_to_cta(ptx::smem_addr(&bar->next_empty[slot]), 0));
        if (++slot == 2) { slot = 0; phase ^= 1u; }
        unit = x >> 1;
        return x >= 0;
    }
};

// Asks for the next unit (whole warp of the leader); false on an expired wait.
struct Asker {
    uint32_t slot = 0, phase = 0;

    __device__ __forceinline__ bool ask(PairBarriers* bar, const volatile int* abort,
                                        uint64_t limit) {
        if (!__all_sync(0xffffffffu,
                        ptx::mbar_wait(&bar->next_empty[slot], phase ^ 1u, abort, limit)))
            return false;
        if ((threadIdx.x & 31) == 0) {
            ptx::mbar_arrive_expect_tx(&bar->next_full[slot], 16);
            ptx::mbar_arrive_expect_tx_cluster(
                ptx::map_to_cta(ptx::smem_addr(&bar->next_full[slot]), 1), 16);
            ptx::try_cancel_cluster(&bar->next[slot], &bar->next_full[slot]);
        }
        __syncwarp();
        if (++slot == 2) { slot = 0; phase ^= 1u; }
        return true;
    }
};

// Set-up of a pair: barriers and tensor memory.  stage_arrivals: arrivals that
// complete a stage's full barrier; walkers: warps of the pair that walk the
// units; side_readers: arrivals on a side slot's empty barrier.
__device__ __forceinline__ void pair_setup(PairBarriers* bar, int stage_arrivals, int walkers,
                                           int side_readers, const CUtensorMap* a,
                                           const CUtensorMap* b) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bar->full[s], stage_arrivals);
            ptx::mbar_init(&bar->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bar->acc_full[i], 1);
            ptx::mbar_init(&bar->acc_empty[i], 16);       // every epilogue warp of the pair
            ptx::mbar_init(&bar->next_full[i], 1);
            ptx::mbar_init(&bar->next_empty[i], walkers);
        }
        for (int s = 0; s < 8; ++s) {
            ptx::mbar_init(&bar->side_full[s], 1);
            ptx::mbar_init(&bar->side_empty[s], side_readers);
        }
        ptx::mbar_init(&bar->drain, 1);
        bar->abort = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(a);
        ptx::tma_prefetch_desc(b);
    }
    if (threadIdx.x >> 5 == 1) {
        ptx::tmem_alloc<2>(&bar->tmem_base, 512);
        ptx::tmem_relinquish<2>();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    ptx::grid_launch_dependents();
}

__device__ __forceinline__ void pair_teardown(uint32_t tmem) {
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (threadIdx.x >> 5 == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc<2>(tmem, 512);
    }
}

__device__ __forceinline__ uint32_t pack16(uint32_t lo, uint32_t hi, bool f16) {
    return f16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// The 32 rows x 64 bytes of a warp's staging leave for rows of `pitch` bytes
// at `out`, as 16-byte pieces where `vec` and the piece is whole, else
// element by element; rows and cols are what may be written.
template <typename E>
__device__ __forceinline__ void copy_staging(const uint8_t* box, E* out, int64_t ld, int rows,
                                             int cols, bool vec) {
    constexpr int PER = 16 / static_cast<int>(sizeof(E));
    const int lane = threadIdx.x & 31;
    const int piece = (lane & 3) * PER;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        if (r >= rows) break;
        const uint8_t* from = box + r * kStagePitch + (lane & 3) * 16;
        E* at = out + r * ld + piece;
        if (vec && piece + PER <= cols) {
            *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(from);
        } else {
            for (int j = 0; j < PER; ++j)
                if (piece + j < cols) at[j] = reinterpret_cast<const E*>(from)[j];
        }
    }
}

}  // namespace
}  // namespace tiles

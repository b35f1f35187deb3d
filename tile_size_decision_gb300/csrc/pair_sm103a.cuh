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
// Epilogue staging, per warp: a box of 32 rows of 64 bytes in the 64-byte
// swizzle of a tensor map (16-byte piece q of row r sits at q ^ (r/2 % 4)), so
// that eight accesses to successive rows hit distinct banks.
constexpr int kBoxBytes = 32 * 64;
constexpr int kStagingBytes = 8 * kBoxBytes;
constexpr int kBarrierBytes = 768;
constexpr int kSideSlots = 16;
// Answers about the next unit that are kept: the loads can be two units ahead of
// the epilogue, whose warps free an answer last, as short units need.
constexpr int kAnswers = 3;

struct PairBarriers {
    uint64_t full[kStages], empty[kStages], acc_full[4], acc_empty[4];
    uint64_t side_full[kSideSlots], side_empty[kSideSlots];   // scales (8-bit), ragged ends (gradient)
    uint64_t drain;
    uint64_t next_full[kAnswers], next_empty[kAnswers];
    ulonglong2 next[kAnswers];                        // answers about the next unit
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(PairBarriers) <= kBarrierBytes, "barrier block too large");

// The pair's units in turn: its own, then those of clusters that have not
// started yet, which a warp of the leader claims a unit or two ahead.  Every role's warp walks through the
// same answers.  (The units are uneven where groups
// are: a fixed assignment left pairs idle for a fifth of the time on the
// weight gradient of 16 uneven groups.)  The answers come in no promised order.
// A walk may end at the first one past the last unit all the same: each is
// awaited before the next is asked for, so no later one is lost, and clusters
// that nobody claimed start by themselves.
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
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            ptx::mbar_arrive_remote(ptx::map_to_cta(ptx::smem_addr(&bar->next_empty[slot]), 0));
        if (++slot == kAnswers) { slot = 0; phase ^= 1u; }
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
            // The walkers' reads of the last answer here come before the
            // async proxy's write of the next.
            ptx::fence_proxy_async();
            ptx::mbar_arrive_expect_tx(&bar->next_full[slot], 16);
            ptx::mbar_arrive_expect_tx_cluster(
                ptx::map_to_cta(ptx::smem_addr(&bar->next_full[slot]), 1), 16);
            ptx::try_cancel_cluster(&bar->next[slot], &bar->next_full[slot]);
        }
        __syncwarp();
        if (++slot == kAnswers) { slot = 0; phase ^= 1u; }
        return true;
    }
};

// An accumulator goes back to the leader's MMA warp (lane 0 of a warp).
__device__ __forceinline__ void hand_back(uint64_t* acc_empty, bool leader) {
    if (leader) ptx::mbar_arrive(acc_empty);
    else ptx::mbar_arrive_remote(ptx::map_to_cta(ptx::smem_addr(acc_empty), 0));
}

// Set-up of a pair: barriers and tensor memory.  stage_arrivals: arrivals that
// complete a stage's full barrier; walkers: warps of the pair that walk the
// units; readers: epilogue warps of a CTA.
__device__ __forceinline__ void pair_setup(PairBarriers* bar, int stage_arrivals, int walkers,
                                           int readers, const CUtensorMap* a,
                                           const CUtensorMap* b) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bar->full[s], stage_arrivals);
            ptx::mbar_init(&bar->empty[s], 1);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(&bar->acc_full[i], 1);
            ptx::mbar_init(&bar->acc_empty[i], 2 * readers);
        }
        for (int i = 0; i < kAnswers; ++i) {
            ptx::mbar_init(&bar->next_full[i], 1);
            ptx::mbar_init(&bar->next_empty[i], walkers);
        }
        for (int s = 0; s < kSideSlots; ++s) {
            ptx::mbar_init(&bar->side_full[s], 1);
            ptx::mbar_init(&bar->side_empty[s], readers);
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

__device__ __forceinline__ uint32_t box_piece(int row, int piece) {
    return static_cast<uint32_t>(row * 64 + ((piece ^ (row >> 1 & 3)) << 4));
}

// The previous box has left: the warp may write the next.
__device__ __forceinline__ void box_begin() {
    if ((threadIdx.x & 31) == 0) ptx::bulk_wait_read_all();
    __syncwarp();
}

// The warp's box leaves for columns x .. and rows y .. of item z of c: whole
// boxes through one TMA store (clipped at the tensor's edges), a ragged
// group's last rows, columns that end inside 16 bytes (a store clips to those,
// not to the element), or a c that TMA cannot address, through the registers.
// `out` is the box's first element, and rows x cols what may be written.
template <typename E>
__device__ __forceinline__ void box_end(const CUtensorMap* map, bool tma, const uint8_t* box, int x,
                                        int y, int z, E* out, int64_t ld, int rows, int cols,
                                        bool whole_rows) {
    constexpr int PER = 16 / static_cast<int>(sizeof(E));
    const int lane = threadIdx.x & 31;
    if (tma && (whole_rows || rows >= 32) && (cols >= 4 * PER || cols % PER == 0)) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            ptx::tma_store_3d(map, box, x, y, z);
            ptx::bulk_commit_group();
        }
        return;
    }
    __syncwarp();
    const int first = (lane & 3) * PER;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        if (r >= rows) break;
        const uint8_t* from = box + box_piece(r, lane & 3);
        E* at = out + r * ld + first;
        if (tma && first + PER <= cols) {
            *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(from);
        } else {
            for (int j = 0; j < PER; ++j)
                if (first + j < cols) at[j] = reinterpret_cast<const E*>(from)[j];
        }
    }
}

}  // namespace
}  // namespace tiles

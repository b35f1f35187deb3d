// Weight gradients of the grouped product: dw[g] = a_g^T x dc_g, where a_g
// and dc_g are the rows of group g (rows x k and rows x n).
//
// The contraction runs over a group's rows, so both operands are MN-major in
// shared memory (their rows are the MMA's K), and a group's last K block ends
// inside a tile: the rows after it belong to the next group.  The MMA warp
// clears them in both operands (a product with another group's infinity or
// NaN would not be zero) and issues only the 16-row steps that hold rows.
//
// One CTA per 128 x 256 tile of one group's gradient; roles as in the GEMM.
#include "product_sm103a.cuh"

namespace tiles {
namespace {

constexpr int kThreads = 192;
constexpr int kStages = 4;
constexpr int kAtomBytes = 64 * 128;                  // 64 rows x 64 columns
constexpr int kABytes = 2 * kAtomBytes, kBBytes = 4 * kAtomBytes;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kSmemBytes = kStages * kStageBytes + kSmemBarrierBytes + kSmemAlignSlack;
constexpr int kTileK = 128, kTileN = 256;

struct Barriers {
    uint64_t full[kStages], empty[kStages], acc_full, drain;
    uint32_t tmem_base;
    int abort;
};

__global__ void __launch_bounds__(kThreads)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const WgradArgs args) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t* base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    Barriers* bar = reinterpret_cast<Barriers*>(base + kStages * kStageBytes);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    int unit = static_cast<int>(blockIdx.x);
    const int per_group = args.k_blocks * args.n_blocks;
    const int group = unit / per_group;
    unit -= group * per_group;
    const int n0 = unit / args.k_blocks * kTileN, k0 = unit % args.k_blocks * kTileK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bar->full[s], 1);
            ptx::mbar_init(&bar->empty[s], 1);
        }
        ptx::mbar_init(&bar->acc_full, 1);
        ptx::mbar_init(&bar->drain, 1);
        bar->abort = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&tmA);
        ptx::tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        ptx::tmem_alloc<1>(&bar->tmem_base, kTileN);
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    const uint32_t tmem = bar->tmem_base;
    volatile int* abort = &bar->abort;
    const uint64_t limit = args.wait_limit_ns;
    const int lo = clamp_offset(args.offsets[group], args.m);
    const int rows = max(0, clamp_offset(args.offsets[group + 1], args.m) - lo);
    const int blocks = (rows + 63) / 64;
    // Columns of dc this tile has, in 64-column atoms.
    const int atoms = min(4, (args.n - n0 + 63) / 64);

    if (warp == 0) {
        uint32_t stage = 0, phase = 0;
        for (int b = 0; b < blocks; ++b) {
            if (!__all_sync(0xffffffffu,
                            ptx::mbar_wait(&bar->empty[stage], phase ^ 1u, abort, limit))) {
                if (lane == 0) raise_error(args.err, abort, kErrProducer);
                settle_after_abort();
                break;
            }
            const bool planted = blockIdx.x == 0 && b == args.drop_stage;
            if (!planted && ptx::elect_one_sync()) {
                uint8_t* at = base + stage * kStageBytes;
                ptx::mbar_arrive_expect_tx(&bar->full[stage], kABytes + atoms * kAtomBytes);
                for (int j = 0; j < 2; ++j)
                    ptx::tma_load_3d(at + j * kAtomBytes, &tmA, &bar->full[stage], k0 + j * 64,
                                     lo + b * 64, 0);
                for (int j = 0; j < atoms; ++j)
                    ptx::tma_load_3d(at + kABytes + j * kAtomBytes, &tmB, &bar->full[stage],
                                     n0 + j * 64, lo + b * 64, 0);
            }
            __syncwarp();
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
    } else if (warp == 1) {
        uint32_t stage = 0, phase = 0;
        const uint32_t saddr = ptx::smem_addr(base);
        const uint64_t a0 = ptx::smem_desc_sw128(saddr, kAtomBytes, 1024);
        const uint64_t b0 = ptx::smem_desc_sw128(saddr + kABytes, kAtomBytes, 1024);
        const bool issuer = ptx::elect_one_sync();
        for (int b = 0; b < blocks; ++b) {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->full[stage], phase, abort, limit))) {
                if (lane == 0) raise_error(args.err, abort, kErrMma);
                break;
            }
            ptx::tc_fence_after();
            const int here = min(64, rows - b * 64);
            const int steps = (here + 15) / 16;
            if (here < steps * 16) {
                // Rows here .. 16*steps-1 of every atom: 8 pieces of 16 bytes
                // each.  The swizzle stays inside a row, so its order does
                // not matter.
                const uint32_t st = saddr + stage * kStageBytes;
                const int pieces = (steps * 16 - here) * 8;
                for (int j = 0; j < 2 + atoms; ++j)
                    for (int p = lane; p < pieces; p += 32)
                        ptx::st_shared_v4(st + j * kAtomBytes + here * 128 + p * 16, 0, 0, 0, 0);
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            if (issuer) {
                const uint64_t sd = (stage * kStageBytes) >> 4;
                for (int kk = 0; kk < steps; ++kk)
                    ptx::mma_f16<1>(tmem, a0 + sd + kk * (2048 >> 4), b0 + sd + kk * (2048 >> 4),
                                    args.idesc, b != 0 || kk != 0);
                ptx::mma_commit<1>(&bar->empty[stage]);
                if (b == blocks - 1) ptx::mma_commit<1>(&bar->acc_full);
            }
            __syncwarp();
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (issuer) {
            ptx::mma_commit<1>(&bar->drain);
            ptx::mbar_wait(&bar->drain, 0, nullptr, limit);
        }
        __syncwarp();
    } else {
        bool ok = true;
        if (blocks > 0) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bar->acc_full, 0, abort, limit));
            if (!ok && lane == 0) raise_error(args.err, abort, kErrEpilogue);
            ptx::tc_fence_after();
        }
        const int quarter = warp & 3;
        const int row = k0 + quarter * 32 + lane;
        const int out_bytes = args.out_dtype == TILES_F32 ? 4 : 2;
        char* out = static_cast<char*>(args.dw) +
                    (static_cast<int64_t>(group) * args.stride_dw +
                     static_cast<int64_t>(row) * args.lddw) * out_bytes;
        // 16-byte stores where every row of every group starts on 16 bytes.
        const bool vec = (reinterpret_cast<uintptr_t>(args.dw) & 15u) == 0 &&
                         args.lddw * out_bytes % 16 == 0 && args.stride_dw * out_bytes % 16 == 0;
#pragma unroll 1
        for (int c = 0; ok && c < atoms * 2; ++c) {
            uint32_t v[32];
            if (blocks > 0) {
                ptx::tmem_ld_32cols(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c * 32, v);
                ptx::tmem_ld_wait();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
            }
            if (row < args.k)
                store_row_chunk(out, n0 + c * 32, args.n, v, args.out_dtype, vec);
        }
        ptx::tc_fence_before();
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<1>(tmem, kTileN);
    }
}

}  // namespace

int launch_wgrad(const CUtensorMap& a, const CUtensorMap& dc, const WgradArgs& args,
                 cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(
        wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return static_cast<int>(e);
    WgradArgs g = args;
    g.k_blocks = (args.k + kTileK - 1) / kTileK;
    g.n_blocks = (args.n + kTileN - 1) / kTileN;
    g.idesc = args.idesc | ptx::idesc_f16_f32acc_majors(false, true, true, kTileK, kTileN);
    const int64_t units = static_cast<int64_t>(args.groups) * g.k_blocks * g.n_blocks;
    return launch(wgrad_kernel, dim3(static_cast<unsigned>(units)), dim3(kThreads), kSmemBytes, st,
                  a, dc, g);
}

}  // namespace tiles

// 8-bit products with many rows, on CTA pairs, dense or grouped:
//   c[i][j] = sum over blocks t of 128 of sa[i][t] * sb[j/128][t] * (a[i] . b[j] within t)
//
// The tensor core sums one K block of 128 from zero into one of its TMEM
// buffers (4 MMA steps of 32), and the epilogue warps add it into fp32
// registers, times the two scales.  So every K block is read back from tensor
// memory.  Its read port also feeds the MMA's accumulation: per K block of a
// 128 x 256 half tile, 3 of the 4 steps read the accumulator (384 clocks) and
// the epilogue's loads take 128 clocks in the plain layout (one lane a thread)
// -- together the 512 clocks of the MMAs -- but 512 in the matrix fragment
// layout.  Hence the plain layout, and the rows of a on the M side: a thread
// owns a row, and its scale is one register, where rows on the N side would
// need a scale per column from shared memory, which the operands already use.
//
// A pair's tile is 256 rows (128 a CTA) by args.tile_cols weight rows (a
// multiple of 32, half of them loaded by each CTA).  Wide tiles (up to 256) have
// two buffers in tensor memory, narrow ones (up to 128) four; the host picks
// the width and with it the kernel (for few tiles the narrow one: 1024 x 1024 x
// 4096 14.1 us against 19.8, while 4096^3 takes 75.5 against 67.9).
//
// Roles (384 threads): warp 0 TMA, warp 1 MMA (leader), warp 2 scales (a small
// ring in shared memory, filled by asynchronous copies ten K blocks ahead), warp
// 3 the units, warps 4-11 epilogue: rows 32*(warp%4), 64-column chunks in turn between the
// two sets.
//
// The reading back bounds it: a K block of a wide tile takes about 860 clocks
// (512 of them MMA), of a narrow one 570 (256).  The epilogue warps never wait
// for a sum; of their time some 250 clocks a K block go to the two waits, the
// scales and the first load, the rest to loads and additions.  4096^3 67.9 us
// (54% of twice the 16-bit rate), 8192 rows in 32 uneven groups by 4096 x 2048
// 88 us (55% of the DRAM floor).  Slower when measured: halves of a tile handed
// over apart (102 us on the groups), 16 epilogue warps (75 on 4096^3), wider
// TMEM loads (72 to 96), scales through registers (79), tiles of one CTA (67
// and 89).
#include "pair_sm103a.cuh"

namespace tiles {
namespace {

constexpr int kScaleSlots = kSideSlots;
// K blocks whose scales are on their way in.  The scale warp walks the units
// that much ahead of the epilogue, and no role gets more than kAnswers units
// ahead of another: with few K blocks a unit it must not wait for more.
constexpr int kScaleLag = 10, kScaleLagShort = 2;
constexpr int kSlotFloats = 128 + 8;                  // 128 rows, 8 chunks of 32 columns
constexpr int kScaleBytes = kScaleSlots * kSlotFloats * 4;
constexpr int kSmemBytes = kStages * kStageBytes + kStagingBytes + kScaleBytes + kBarrierBytes +
                           kSmemAlignSlack;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
static_assert(kScaleBytes % 16 == 0, "the barriers follow the scales");
constexpr int BK = 128;
// Registers a thread.  The block is launched with 168 (384 x 168 = 64512); the
// epilogue holds 128 sums (64 of the narrow tile's) and gets what the service
// warps do not need.
template <int WIDTH> constexpr int kServiceRegisters = WIDTH == 256 ? 96 : 80;
template <int WIDTH> constexpr int kEpilogueRegisters = WIDTH == 256 ? 200 : 208;
static_assert(128 * kServiceRegisters<256> + 256 * kEpilogueRegisters<256> <= kThreads * 168 &&
              128 * kServiceRegisters<128> + 256 * kEpilogueRegisters<128> <= kThreads * 168,
              "registers");

struct Unit {
    int group;
    int n0, width;     // first weight row, and TMEM columns
    int row0, end;
};

struct Units {
    RowTileCursor cursor;

    __device__ __forceinline__ bool get(int u, const ProductArgs& a, Unit* out) {
        const int tile = u / a.n_blocks;
        out->n0 = (u - tile * a.n_blocks) * a.tile_cols;
        out->width = (min(a.tile_cols, a.n - out->n0) + 31) / 32 * 32;
        RowTile rt;
        if (a.groups > 0) {
            if (!cursor.seek(a.offsets, a.groups, a.m, 256, tile, &rt)) return false;
        } else {
            rt = RowTile{0, tile * 256, a.m};
            if (rt.row0 >= a.m) return false;
        }
        out->group = rt.group;
        out->row0 = rt.row0;
        out->end = min(rt.end, rt.row0 + 256);
        return true;
    }
};

template <int WIDTH>
__global__ void __launch_bounds__(kThreads, 1)
    pair8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                 const __grid_constant__ CUtensorMap tmC, const ProductArgs args) {
    constexpr int BUFFERS = 512 / WIDTH, HALVES = WIDTH / 128;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t* base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* staging = base + kStages * kStageBytes;
    float* scales = reinterpret_cast<float*>(staging + kStagingBytes);
    PairBarriers* bar = reinterpret_cast<PairBarriers*>(staging + kStagingBytes + kScaleBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = static_cast<int>(blockIdx.x) / 2;
    Walk walk{pair};
    Units units;
    Unit un;

    // The grid is the host's upper bound: clusters past the last unit leave.
    ptx::grid_dependency_wait();
    if (!units.get(pair, args, &un)) return;
    const uint64_t limit = wait_limit(args);
    // Walkers: both TMA and scale warps, every epilogue warp, the MMA warp and
    // the asking warp.
    pair_setup(bar, 1, 2 + 2 + 16 + 1 + 1, 8, &tmW, &tmA);

    const uint32_t tmem = bar->tmem_base;
    volatile int* abort = &bar->abort;
    const int blocks = args.k_blocks;
    bool failed = false;

    if (warp < 4) {
        ptx::registers_dec<kServiceRegisters<WIDTH>>();
        if (warp == 0) {
            // ---------------- TMA producer ----------------
            uint32_t stage = 0, phase = 0;
            int issued = 0;
            const bool issuer = ptx::elect_one_sync();
            const uint32_t full0 = ptx::map_to_cta(ptx::smem_addr(&bar->full[0]), 0);
            // (A box of half a tile's weight rows, also where the last tile has fewer.)
            const uint32_t both = 2u * static_cast<uint32_t>(kHalfBytes + args.tile_cols / 2 * 128);
            do {
                const int first = un.n0 + static_cast<int>(rank) * (un.width / 2);
                const int row0 = un.row0 + static_cast<int>(rank) * 128;
                for (int b = 0; b < blocks; ++b) {
                    if (!__all_sync(0xffffffffu,
                                    ptx::mbar_wait(&bar->empty[stage], phase ^ 1u, abort, limit))) {
                        failed = true;
                        break;
                    }
                    const bool planted = pair == 0 && issued == args.drop_stage;
                    if (!planted && issuer) {
                        uint8_t* a = base + stage * kStageBytes;
                        const uint32_t fb = full0 + stage * 8;
                        if (leader) ptx::mbar_arrive_expect_tx(&bar->full[stage], both);
                        ptx::tma_load_3d_pair(a, &tmA, fb, b * BK, row0, 0);
                        ptx::tma_load_3d_pair(a + kHalfBytes, &tmW, fb, b * BK, first, un.group);
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            } while (!failed && walk.next(bar, abort, limit, &failed) &&
                     units.get(walk.unit, args, &un));
            if (failed) {
                if (lane == 0) raise_error(args.err, abort, kErrProducer);
                settle_after_abort();
            }
        } else if (warp == 1 && leader) {
            // ---------------- MMA issuer ----------------
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            const uint32_t sA = ptx::smem_addr(base);
            const uint64_t a0 = ptx::smem_desc_sw128(sA, 16, 1024);
            const uint64_t w0 = ptx::smem_desc_sw128(sA + kHalfBytes, 16, 1024);
            const bool issuer = ptx::elect_one_sync();
            do {
                const uint32_t idesc = args.idesc | static_cast<uint32_t>(un.width >> 3) << 17;
                for (int b = 0; b < blocks; ++b) {
                    // The accumulator comes last: its return is what a K block
                    // usually waits for.
                    const bool ok = ptx::mbar_wait(&bar->full[stage], phase, abort, limit) &&
                                    ptx::mbar_wait(&bar->acc_empty[acc], acc_phase ^ 1u, abort, limit);
                    if (!__all_sync(0xffffffffu, ok)) {
                        failed = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (issuer) {
                        const uint64_t at = (stage * kStageBytes) >> 4;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_f8<2>(tmem + acc * WIDTH, a0 + at + kk * 2, w0 + at + kk * 2,
                                           idesc, kk != 0);
                        ptx::mma_commit<2>(&bar->empty[stage]);
                        ptx::mma_commit<2>(&bar->acc_full[acc]);
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                    acc = (acc + 1) % BUFFERS;
                acc_phase ^= acc == 0;
                }
            } while (!failed && walk.next(bar, abort, limit, &failed) &&
                     units.get(walk.unit, args, &un));
            if (failed && lane == 0) raise_error(args.err, abort, kErrMma);
            if (issuer) {
                ptx::mma_commit_local<2>(&bar->drain);
                ptx::mbar_wait(&bar->drain, 0, nullptr, limit);
            }
            __syncwarp();
        } else if (warp == 3 && leader) {
            // ---------------- the next units ----------------
            Asker asker;
            do {
                if (!asker.ask(bar, abort, limit)) {
                    failed = true;
                    break;
                }
            } while (walk.next(bar, abort, limit, &failed) && units.get(walk.unit, args, &un));
            if (failed) {
                if (lane == 0) raise_error(args.err, abort, kErrProducer);
                settle_after_abort();
            }
        } else if (warp == 2) {
            // ---------------- scales ----------------
            // Asynchronous copies into the ring, `lag` K blocks ahead of
            // the slot that is handed on (across units).  Scales of rows past
            // the end are not copied: their sums are never written.
            uint32_t slot = 0, phase = 0, done = 0;
            int pending = 0;
            const int lag = 2 * blocks >= kScaleLag ? kScaleLag : kScaleLagShort;
            do {
                const int row0 = un.row0 + static_cast<int>(rank) * 128 + lane;
                const float* sa = args.sa + row0 * args.sa_row;
                // Lane c < 8: the weight's scale of column chunk c.
                const float* sb = args.sb + un.group * args.sb_group +
                                  (min(un.n0 + (lane & 7) * 32, args.n - 1) / kScaleBlock) * args.sb_row;
                for (int b = 0; b < blocks; ++b) {
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->side_empty[slot], phase ^ 1u,
                                                                abort, limit))) {
                        failed = true;
                        break;
                    }
                    float* to = scales + slot * kSlotFloats + lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (row0 + i * 32 < un.end) ptx::cp_async_4(to + i * 32, sa + i * 32 * args.sa_row);
                    if (lane < 8) ptx::cp_async_4(to + 128, sb);
                    ptx::cp_async_commit();
                    sa += args.sa_block;
                    sb += args.sb_block;
                    if (++slot == kScaleSlots) { slot = 0; phase ^= 1u; }
                    if (++pending > lag) {
                        if (lag == kScaleLag) ptx::cp_async_wait_groups<kScaleLag>();
                        else ptx::cp_async_wait_groups<kScaleLagShort>();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&bar->side_full[done]);
                        done = (done + 1) % kScaleSlots;
                        --pending;
                    }
                }
            } while (!failed && walk.next(bar, abort, limit, &failed) &&
                     units.get(walk.unit, args, &un));
            ptx::cp_async_wait_groups<0>();
            __syncwarp();
            for (; pending > 0; --pending) {
                if (lane == 0) ptx::mbar_arrive(&bar->side_full[done]);
                done = (done + 1) % kScaleSlots;
            }
            if (failed && lane == 0) raise_error(args.err, abort, kErrEpilogue);
        }
    } else {
        // ---------------- epilogue ----------------
        ptx::registers_inc<kEpilogueRegisters<WIDTH>>();
        const int quarter = warp & 3, set = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* box = staging + (warp - 4) * kBoxBytes;
        const bool f16 = args.c_dtype == TILES_F16;
        // One 64-byte row of the box, from 16 words.
        auto fill = [&](const uint32_t (&w)[16]) {
            box_begin();
            const uint32_t at = ptx::smem_addr(box);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                ptx::st_shared_v4(at + box_piece(lane, q), w[4 * q], w[4 * q + 1], w[4 * q + 2],
                                  w[4 * q + 3]);
        };
        uint32_t acc = 0, acc_phase = 0, slot = 0, slot_phase = 0;
        // The leader's acc_empty barriers.
        const uint32_t acc_empty = ptx::map_to_cta(ptx::smem_addr(&bar->acc_empty[0]), 0);
        do {
            // This thread's row: columns 64 * (2h + set) + 32q + .. in
            // sum[2h + q], as pairs.
            uint64_t sum[2 * HALVES][16];
#pragma unroll
            for (int j = 0; j < 2 * HALVES; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[j][i] = 0;
            // 16 columns at a time, the next ones' load in flight while these are
            // added; the first of the next K block's too, so that its waits
            // and the first load's latency are behind the last additions.
            // (Columns past the width hold old sums that nothing reads.)
            constexpr int PARTS = 4 * HALVES;
            auto column = [](int i) { return (i >> 2) * 128 + (i & 3) * 16; };
            uint32_t v[2][16];
            float scale[2 * HALVES], next[2 * HALVES];     // row's times chunk's
            uint32_t t = 0;
            // Waits for the next K block, reads its scales into `to` and starts
            // the load of its first columns.
            auto open = [&](float (&to)[2 * HALVES]) {
                bool ok = ptx::mbar_wait(&bar->side_full[slot], slot_phase, abort, limit);
                const float* sc = scales + slot * kSlotFloats;
                const float row_scale = sc[quarter * 32 + lane];
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const float2 w = *reinterpret_cast<const float2*>(sc + 128 + 4 * h + set * 2);
                    to[2 * h] = row_scale * w.x;
                    to[2 * h + 1] = row_scale * w.y;
                }
                ok = ok && ptx::mbar_wait(&bar->acc_full[acc], acc_phase, abort, limit);
                if (!__all_sync(0xffffffffu, ok)) return false;
                if (lane == 0) ptx::mbar_arrive(&bar->side_empty[slot]);
                if (++slot == kScaleSlots) { slot = 0; slot_phase ^= 1u; }
                ptx::tc_fence_after();
                t = tmem + lanes + acc * WIDTH + set * 64;
                ptx::tmem_ld_16cols(t, v[0], 0);
                return true;
            };
            if (!open(scale)) {
                failed = true;
                break;
            }
            auto add = [&](int i) {
                const uint32_t s = __float_as_uint(scale[i >> 1]);
                const uint64_t ss = ptx::pack_pair(s, s);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    ptx::fma_pair(sum[i >> 1][(i & 1) * 8 + q],
                                  ptx::pack_pair(v[i & 1][2 * q], v[i & 1][2 * q + 1]), ss);
            };
#pragma unroll 1
            for (int b = 0; b < blocks; ++b) {
                ptx::tmem_ld_wait_for(v[0]);
#pragma unroll
                for (int i = 0; i + 1 < PARTS; ++i) {
                    ptx::tmem_ld_16cols(t + column(i + 1), v[(i + 1) & 1], 0);
                    add(i);
                    ptx::tmem_ld_wait_for(v[(i + 1) & 1]);
                }
                // All read: back to the MMA before the last sums.
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_remote(acc_empty + acc * 8);
                acc = (acc + 1) % BUFFERS;
                acc_phase ^= acc == 0;
                if (b + 1 < blocks && !open(next)) {
                    failed = true;
                    break;
                }
                add(PARTS - 1);
#pragma unroll
                for (int i = 0; i < 2 * HALVES; ++i) scale[i] = next[i];
            }
            if (failed) break;
            const int row0 = un.row0 + static_cast<int>(rank) * 128 + quarter * 32;
            const int rows = un.end - row0;                // what is left to write
#pragma unroll
            for (int j = 0; j < 2 * HALVES; ++j) {
                const int col0 = un.n0 + (j >> 1) * 128 + set * 64 + (j & 1) * 32;
                const int cols = min(args.n, un.n0 + un.width) - col0;
                if (rows <= 0 || cols <= 0) break;
                const int64_t out0 = static_cast<int64_t>(row0) * args.ldc + col0;
                uint32_t v[2][16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    ptx::unpack_pair(sum[j][i], v[i >> 3][2 * (i & 7)], v[i >> 3][2 * (i & 7) + 1]);
                if (args.c_dtype == TILES_F32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        fill(v[h]);
                        if (cols > h * 16)
                            box_end(&tmC, args.tma_store, box, col0 + h * 16, row0, 0,
                                    static_cast<float*>(args.c) + out0 + h * 16, args.ldc, rows,
                                    cols - h * 16, false);
                    }
                } else {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        p[i] = pack16(v[i >> 3][2 * (i & 7)], v[i >> 3][2 * (i & 7) + 1], f16);
                    fill(p);
                    box_end(&tmC, args.tma_store, box, col0, row0, 0,
                            static_cast<uint16_t*>(args.c) + out0, args.ldc, rows, cols, false);
                }
            }
        } while (walk.next(bar, abort, limit, &failed) && units.get(walk.unit, args, &un));
        if (failed && lane == 0) raise_error(args.err, abort, kErrEpilogue);
        box_begin();                                       // the last box has been read
    }
    pair_teardown(tmem);
}

}  // namespace

int pair_max_groups(int sms) {
    if (cudaFuncSetAttribute(pair8_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes) != cudaSuccess) {
        cudaGetLastError();
        return sms / 2;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, pair8_kernel<256>, &cfg) != cudaSuccess ||
        clusters <= 0) {
        cudaGetLastError();
        return sms / 2;
    }
    return clusters;
}

namespace {

template <int WIDTH>
int launch_width(const CUtensorMap& w, const CUtensorMap& a, const CUtensorMap& c,
                 const ProductArgs& args, int units, cudaStream_t st) {
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(pair8_kernel<WIDTH>, kSmemBytes, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    return launch_cluster(pair8_kernel<WIDTH>, 2, dim3(static_cast<unsigned>(2 * units)),
                          dim3(kThreads), kSmemBytes, st, w, a, c, args);
}

}  // namespace

int launch_pair8(const CUtensorMap& weight, const CUtensorMap& rows, const CUtensorMap& out,
                 const ProductArgs& args, int units, cudaStream_t st) {
    return args.tile_cols > 128 ? launch_width<256>(weight, rows, out, args, units, st)
                                : launch_width<128>(weight, rows, out, args, units, st);
}

}  // namespace tiles

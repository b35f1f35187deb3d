// Products of a few rows with a weight: c[rows, n] = a[rows, k] x weight.
//
// The weight is the large operand, so it takes the MMA's M side: a tile is
// 128 weight columns (TMEM lanes) by NT rows of a (TMEM columns, the MMA's N,
// whose granularity of 16 fits a ragged group's few rows).  Each weight
// element is read once and used for all NT rows, so with few rows the kernel
// is bound by streaming the weight from DRAM; the shared memory of a block is
// kept under half an SM's, so that two resident blocks keep loads in flight
// while one of them starts or ends.
//
// When there are fewer (row tile, weight block) units than SMs, `split` CTAs
// of a cluster take a share of K each.  They leave their fp32 partial tiles in
// shared memory, and each then adds one share of the columns over the
// cluster, in rank order, and stores it: no atomics, the same bits each run.
//
// e4m3 operands: the tensor core sums one block of 128 along K from zero; the
// epilogue warps add it, times the row's and the weight block's scale, into
// fp32 registers (two TMEM buffers, so that the next block's MMAs overlap).
//
// Roles as in the GEMM: warp 0 TMA, warp 1 MMA, warps 2-5 epilogue.
//
// 64 rows over 15 of 16 groups, 2048 x 2048 bf16 weights (126 MB): 22.8 us, 82%
// of the measured copy bandwidth.  16 rows by a 4096 x 4096 e4m3 weight: 7.5 us
// where the weight's bytes take 2.5 (5.4 with the weight in L2); the rest is the
// chain of one CTA's loads, K blocks and the cluster's addition, as latency.
#include "product_sm103a.cuh"

namespace tiles {
namespace {

constexpr int kThreads = 192;
constexpr int kRowBytes = 128;                        // one K block of a row
constexpr int kWeightBytes = 128 * kRowBytes;         // 16 KB a stage
constexpr int kScaleChunk = 16;                       // K blocks whose scales sit in shared memory

struct Barriers {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int abort;
    int group, row0, end, found;
};
static_assert(sizeof(Barriers) <= kSmemBarrierBytes, "barrier block too large");

template <int KIND, int NT>
struct StreamLayout {
    static constexpr int STAGES = NT == 16 ? 6 : NT == 32 ? 5 : 4;
    static constexpr int ROWS_BYTES = NT * kRowBytes;
    static constexpr int STAGE_BYTES = kWeightBytes + ROWS_BYTES;
    static constexpr int SCALE_BYTES = KIND == kWeight8NK ? NT * kScaleChunk * 4 : 0;
    static constexpr int SMEM_BYTES =
        STAGES * STAGE_BYTES + SCALE_BYTES + kSmemBarrierBytes + kSmemAlignSlack;
    static constexpr int BUFFERS = KIND == kWeight8NK ? 2 : 1;
    static constexpr int COLS = NT * BUFFERS;
    static constexpr int TMEM_COLS = COLS < 32 ? 32 : COLS;
    static_assert(NT * 128 * 4 <= STAGES * STAGE_BYTES, "a partial tile must fit the stages");
    static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two blocks per SM");
    static_assert(2 * TMEM_COLS <= 512, "two blocks' tensor memory");
};

// Columns rank * NT/S .. of the cluster's partial tiles, added in rank order
// and stored: this thread's weight column, at `mine` in every CTA.  A read from
// another CTA's shared memory takes a third of a microsecond, so 32 of them
// are in flight at once.
template <int S, int NT>
__device__ __forceinline__ void add_shares(uint32_t mine, int rank, int rows, void* c, int64_t at,
                                           int64_t ldc, bool in, int dtype) {
    constexpr int PER = NT / S, BATCH = 32 / S < PER ? 32 / S : PER;
    uint32_t from[S];
#pragma unroll
    for (int s = 0; s < S; ++s) from[s] = ptx::map_to_cta(mine, s);
    for (int c0 = rank * PER; c0 < (rank + 1) * PER && c0 < rows; c0 += BATCH) {
        float x[S][BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
#pragma unroll
            for (int s = 0; s < S; ++s)
                x[s][j] = ptx::ld_shared_cluster(from[s] + static_cast<uint32_t>(c0 + j) * 512u);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            float v = x[0][j];
#pragma unroll
            for (int s = 1; s < S; ++s) v += x[s][j];
            if (in && c0 + j < rows) store_one(c, at + (c0 + j) * ldc, v, dtype);
        }
    }
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kThreads)
    stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                  const ProductArgs args) {
    using L = StreamLayout<KIND, NT>;
    constexpr int STAGES = L::STAGES;
    constexpr int BK = KIND == kWeight8NK ? 128 : 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t* base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* smW = base;
    uint8_t* smA = base + STAGES * kWeightBytes;
    float* scales = reinterpret_cast<float*>(base + STAGES * L::STAGE_BYTES);
    Barriers* bar = reinterpret_cast<Barriers*>(base + STAGES * L::STAGE_BYTES + L::SCALE_BYTES);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = args.split;
    const int unit = static_cast<int>(blockIdx.x) / split;
    const int rank = static_cast<int>(blockIdx.x) - unit * split;   // rank in the cluster
    const int row_tile = unit / args.n_blocks;
    const int n0 = (unit - row_tile * args.n_blocks) * 128;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(&bar->full[s], 1);
            ptx::mbar_init(&bar->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&bar->acc_full[b], 1);
            ptx::mbar_init(&bar->acc_empty[b], 4);
        }
        ptx::mbar_init(&bar->drain, 1);
        bar->abort = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&tmW);
        ptx::tma_prefetch_desc(&tmA);
    }
    if (warp == 1) {
        ptx::tmem_alloc<1>(&bar->tmem_base, L::TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    ptx::grid_dependency_wait();
    if (warp == 2) {
        RowTile rt{0, row_tile * NT, args.m};
        bool found = true;
        if (args.groups > 0) {
            RowTileCursor cursor;
            found = cursor.seek(args.offsets, args.groups, args.m, NT, row_tile, &rt);
        }
        if (lane == 0) {
            bar->group = rt.group;
            bar->row0 = rt.row0;
            bar->end = rt.end;
            bar->found = found;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // Only now: the next kernel's blocks must not take the tensor memory that
    // this block still waits for.
    ptx::grid_launch_dependents();

    const uint32_t tmem = bar->tmem_base;
    const int group = bar->group, row0 = bar->row0, end = bar->end;
    volatile int* abort = &bar->abort;
    const uint64_t limit = args.wait_limit_ns;
    const int kb0 = rank * args.k_blocks / split, kb1 = (rank + 1) * args.k_blocks / split;
    float acc[NT];                                  // epilogue threads: one weight column's NT rows

    if (!bar->found) {
        // Past the last row tile (the grid is the host's upper bound): the
        // whole cluster leaves.
    } else if (warp == 0) {
        uint32_t stage = 0, phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu,
                            ptx::mbar_wait(&bar->empty[stage], phase ^ 1u, abort, limit))) {
                if (lane == 0) raise_error(args.err, abort, kErrProducer);
                settle_after_abort();
                break;
            }
            const bool planted = blockIdx.x == 0 && kb == args.drop_stage;
            if (!planted && ptx::elect_one_sync()) {
                ptx::mbar_arrive_expect_tx(&bar->full[stage], L::STAGE_BYTES);
                uint8_t* w = smW + stage * kWeightBytes;
                if constexpr (KIND == kWeight16KN) {
                    ptx::tma_load_3d(w, &tmW, &bar->full[stage], n0, kb * BK, group);
                    ptx::tma_load_3d(w + kWeightBytes / 2, &tmW, &bar->full[stage], n0 + 64,
                                     kb * BK, group);
                } else {
                    ptx::tma_load_3d(w, &tmW, &bar->full[stage], kb * BK, n0, group);
                }
                ptx::tma_load_3d(smA + stage * L::ROWS_BYTES, &tmA, &bar->full[stage], kb * BK,
                                 row0, 0);
            }
            __syncwarp();
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
    } else if (warp == 1) {
        uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
        // The weight, MN-major: 16 K rows = two 8-row groups of 1024 B,
        // 64-column atoms 8 KB apart; K-major: 32 bytes a step inside the
        // swizzled row, 8-row groups 1024 B apart.
        const uint64_t w0 = KIND == kWeight16KN
            ? ptx::smem_desc_sw128(ptx::smem_addr(smW), kWeightBytes / 2, 1024)
            : ptx::smem_desc_sw128(ptx::smem_addr(smW), 16, 1024);
        const uint64_t a0 = ptx::smem_desc_sw128(ptx::smem_addr(smA), 16, 1024);
        constexpr int WSTEP = (KIND == kWeight16KN ? 2048 : 32) >> 4;
        const bool issuer = ptx::elect_one_sync();
        for (int kb = kb0; kb < kb1; ++kb) {
            bool ok = true;
            if constexpr (KIND == kWeight8NK)
                ok = ptx::mbar_wait(&bar->acc_empty[buf], buf_phase ^ 1u, abort, limit);
            ok = ok && ptx::mbar_wait(&bar->full[stage], phase, abort, limit);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) raise_error(args.err, abort, kErrMma);
                break;
            }
            ptx::tc_fence_after();
            if (issuer) {
                const uint64_t w = w0 + ((stage * kWeightBytes) >> 4);
                const uint64_t a = a0 + ((stage * L::ROWS_BYTES) >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if constexpr (KIND == kWeight8NK)
                        ptx::mma_f8<1>(tmem + buf * NT, w + kk * WSTEP, a + kk * 2, args.idesc, kk != 0);
                    else
                        ptx::mma_f16<1>(tmem, w + kk * WSTEP, a + kk * 2, args.idesc,
                                        kb != kb0 || kk != 0);
                }
                ptx::mma_commit<1>(&bar->empty[stage]);
                if (KIND == kWeight8NK || kb == kb1 - 1) ptx::mma_commit<1>(&bar->acc_full[buf]);
            }
            __syncwarp();
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            if constexpr (KIND == kWeight8NK) {
                buf ^= 1u;
                if (buf == 0) buf_phase ^= 1u;
            }
        }
        if (issuer) {
            ptx::mma_commit<1>(&bar->drain);
            ptx::mbar_wait(&bar->drain, 0, nullptr, limit);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t v[NT < 32 ? NT : 32];
        bool ok = true;
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[c] = 0.0f;
        if constexpr (KIND == kWeight8NK) {
            const int t = threadIdx.x - 64;
            const float* sb = args.sb + static_cast<int64_t>(group) * args.sb_group +
                              static_cast<int64_t>(n0 / kScaleBlock) * args.sb_row;
            uint32_t buf = 0, buf_phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int in_chunk = (kb - kb0) % kScaleChunk;
                if (in_chunk == 0) {
                    // The next K blocks' scales, row times weight block.
                    // Every epilogue warp passes here as often, also after
                    // an expired wait, so the barriers always pair up.
                    ptx::named_barrier(1, 128);
                    // (All loads first: one at a time they took a microsecond
                    // each.)
                    constexpr int EACH = kScaleChunk * NT / 128;
                    float r[EACH], w[EACH];
#pragma unroll
                    for (int j = 0; j < EACH; ++j) {
                        const int i = j * 128 + t, row = row0 + i % NT;
                        const int64_t b = min(kb + i / NT, args.k_blocks - 1);
                        r[j] = row < end ? args.sa[row * args.sa_row + b * args.sa_block] : 0.0f;
                        w[j] = sb[b * args.sb_block];
                    }
#pragma unroll
                    for (int j = 0; j < EACH; ++j) scales[j * 128 + t] = r[j] * w[j];
                    ptx::named_barrier(1, 128);
                }
                if (ok) ok = __all_sync(0xffffffffu,
                                        ptx::mbar_wait(&bar->acc_full[buf], buf_phase, abort, limit));
                if (ok) {
                    ptx::tc_fence_after();
                    const float4* sc = reinterpret_cast<const float4*>(scales + in_chunk * NT);
#pragma unroll
                    for (int c = 0; c < NT; c += 32) {
                        if constexpr (NT == 16) {
                            ptx::tmem_ld_16cols(tmem + lanes + buf * NT, v, 0);
                        } else {
                            ptx::tmem_ld_32cols(tmem + lanes + buf * NT + c, v);
                        }
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < (NT < 32 ? NT : 32); i += 4) {
                            const float4 s = sc[(c + i) / 4];
                            acc[c + i] += __uint_as_float(v[i]) * s.x;
                            acc[c + i + 1] += __uint_as_float(v[i + 1]) * s.y;
                            acc[c + i + 2] += __uint_as_float(v[i + 2]) * s.z;
                            acc[c + i + 3] += __uint_as_float(v[i + 3]) * s.w;
                        }
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar->acc_empty[buf]);
                }
                buf ^= 1u;
                if (buf == 0) buf_phase ^= 1u;
            }
        } else {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bar->acc_full[0], 0, abort, limit));
            if (ok) {
                ptx::tc_fence_after();
#pragma unroll
                for (int c = 0; c < NT; c += 32) {
                    if constexpr (NT == 16) ptx::tmem_ld_16cols(tmem + lanes, v, 0);
                    else ptx::tmem_ld_32cols(tmem + lanes + c, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < (NT < 32 ? NT : 32); ++i) acc[c + i] = __uint_as_float(v[i]);
                }
                ptx::tc_fence_before();
            }
        }
        if (!ok && lane == 0) raise_error(args.err, abort, kErrEpilogue);
        // Thread f of the 128 holds weight column n0 + f.
        const int f = (warp & 3) * 32 + lane;
        if (split == 1) {
            if (ok && n0 + f < args.n) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    if (row0 + c < end)
                        store_one(args.c, static_cast<int64_t>(row0 + c) * args.ldc + n0 + f, acc[c],
                                  args.c_dtype);
            }
        } else {
            // The stages are idle: every load has been consumed.
            float* part = reinterpret_cast<float*>(base);
#pragma unroll
            for (int c = 0; c < NT; ++c) part[c * 128 + f] = acc[c];
        }
    }

    if (bar->found && split > 1) {
        ptx::cluster_sync();
        if (warp >= 2 && !*abort) {
            const int f = (warp & 3) * 32 + lane;
            const uint32_t mine = ptx::smem_addr(base) + static_cast<uint32_t>(f) * 4u;
            const int rows = end - row0, col = n0 + f;
            void* c = args.c;
            const int64_t at = static_cast<int64_t>(row0) * args.ldc + col;
            if (split == 2) add_shares<2, NT>(mine, rank, rows, c, at, args.ldc, col < args.n, args.c_dtype);
            else if (split == 4) add_shares<4, NT>(mine, rank, rows, c, at, args.ldc, col < args.n, args.c_dtype);
            else add_shares<8, NT>(mine, rank, rows, c, at, args.ldc, col < args.n, args.c_dtype);
        }
        ptx::cluster_sync();                        // no CTA leaves while another reads from it
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<1>(tmem, L::TMEM_COLS);
    }
}

template <int KIND, int NT>
int launch_one(const CUtensorMap& w, const CUtensorMap& a, const ProductArgs& args, int64_t units,
               cudaStream_t st) {
    using L = StreamLayout<KIND, NT>;
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(stream_kernel<KIND, NT>, L::SMEM_BYTES, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    return launch_cluster(stream_kernel<KIND, NT>, args.split,
                          dim3(static_cast<unsigned>(units * args.split)), dim3(kThreads),
                          L::SMEM_BYTES, st, w, a, args);
}

template <int KIND>
int launch_rows(int tile_rows, const CUtensorMap& w, const CUtensorMap& a, const ProductArgs& args,
                int64_t units, cudaStream_t st) {
    switch (tile_rows) {
        case 16: return launch_one<KIND, 16>(w, a, args, units, st);
        case 32: return launch_one<KIND, 32>(w, a, args, units, st);
        default: return launch_one<KIND, 64>(w, a, args, units, st);
    }
}

}  // namespace

int launch_stream(int kind, int tile_rows, const CUtensorMap& weight, const CUtensorMap& rows,
                  const ProductArgs& args, int64_t units, cudaStream_t st) {
    switch (kind) {
        case kWeight16KN: return launch_rows<kWeight16KN>(tile_rows, weight, rows, args, units, st);
        case kWeight16NK: return launch_rows<kWeight16NK>(tile_rows, weight, rows, args, units, st);
        default: return launch_rows<kWeight8NK>(tile_rows, weight, rows, args, units, st);
    }
}

}  // namespace tiles

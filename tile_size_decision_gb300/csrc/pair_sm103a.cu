// 16-bit products with many rows, on CTA pairs: c[rows, n] = a[rows, k] x weight
// grouped by expert, and the grouped weight gradient.
//
// As in the few-rows kernel the weight takes the MMA's M side: a pair's tile
// is 256 weight columns (128 TMEM lanes in each CTA) by up to 256 rows of a
// (TMEM columns).  The rows are the MMA's N, whose granularity of 32 for a
// pair lets the last tile of a ragged group do only the work it has.  Each CTA
// loads its 128 weight columns and half of the rows, 32 KB per K block of 512
// MMA clocks: 64 B/clk, about what an SM fills from L2, so the pair's sharing
// of the rows is what lets the tensor core run.
//
// The weight gradient dw[g] = a_g^T dc_g is the same tile with other names:
// dc's columns are the MMA's M, a's columns its N, and the group's rows the
// contraction.  Its last K block ends inside a tile; one warp in each CTA
// clears the rows past the group's end in both operands (another group's
// infinity times zero would not be zero) before the MMA reads them.
//
// Roles (384 threads): warp 0 TMA, warp 1 MMA (leader), warp 2 the clearing of
// ragged ends (weight gradient), warp 3 the units (leader), warps 4-11 epilogue:
// lanes 32*(warp%4), column chunks of 32 in turn between the two sets of four.
// The epilogue reads tensor memory in the matrix fragment layout (a quarter of
// the plain layout's rate, one K block's MMA time per tile), because stmatrix
// then transposes it: a row of c is a TMEM column.
//
// The tensor cores bound long contractions, the results' way out short ones.
// 32768 rows in 16 uneven groups, 1024 x 2048 bf16: products and the rows'
// gradient 83 us (88% of the measured rate), the weight gradient 90 (81%), from a
// graph with pauses; called back to back the power cap makes it 95 to 98 and 99
// to 103.  What made the products faster (95 us from a graph): the next units
// asked for by a warp of its own, and a stage's rows in one load (the TMA warp,
// with six loads a stage, had been the slowest role: 650 clocks a K block).
// Measured before that on 30000 x 1024 x 2048 (83.5 us): without the stores
// 74.9, without the transposition 83.9, through registers instead of TMA 84.9,
// with two boxes a warp and the TMEM loads a chunk ahead 84.3.
#include "pair_sm103a.cuh"

namespace tiles {
namespace {

constexpr int kSmemBytes = kStages * kStageBytes + kStagingBytes + kBarrierBytes + kSmemAlignSlack;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
constexpr int BK = 64;

// One unit of work.
struct Unit {
    int group;
    int n0;            // first weight column of the pair's tile
    int row0, end;     // output rows: rows of a, or columns of a (weight gradient)
    int width;         // TMEM columns: rows rounded up to the MMA's N
    int k0, k1;        // contraction range: [0, k), or the group's rows
    int blocks;        // K blocks
};

template <int KIND>
struct Units {
    RowTileCursor cursor;

    __device__ __forceinline__ bool get(int u, const ProductArgs& a, Unit* out) {
        const int tile = u / a.n_blocks;
        out->n0 = (u - tile * a.n_blocks) * 256;
        RowTile rt;
        if constexpr (KIND == kWeightGrad) {
            const int per_group = (a.k + kMaxWidth - 1) / kMaxWidth;
            rt.group = tile / per_group;
            if (rt.group >= a.groups) return false;
            rt.row0 = (tile - rt.group * per_group) * kMaxWidth;
            rt.end = a.k;
            out->k0 = clamp_offset(a.offsets[rt.group], a.m);
            out->k1 = max(out->k0, clamp_offset(a.offsets[rt.group + 1], a.m));
            // Halves of 64-column atoms in each CTA.
            out->width = rt.end - rt.row0 > 128 ? 256 : 128;
        } else {
            if (!cursor.seek(a.offsets, a.groups, a.m, kMaxWidth, tile, &rt)) return false;
            out->k0 = 0;
            out->k1 = a.k;
            rt.end = min(rt.end, rt.row0 + kMaxWidth);
            out->width = (rt.end - rt.row0 + 31) / 32 * 32;
        }
        out->group = rt.group;
        out->row0 = rt.row0;
        out->end = rt.end;
        out->blocks = (out->k1 - out->k0 + BK - 1) / BK;
        return true;
    }
};

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmA128, const __grid_constant__ CUtensorMap tmC,
                const ProductArgs args) {
    constexpr bool GRAD = KIND == kWeightGrad;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t* base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* staging = base + kStages * kStageBytes;
    PairBarriers* bar = reinterpret_cast<PairBarriers*>(staging + kStagingBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = static_cast<int>(blockIdx.x) / 2;
    Walk walk{pair};
    Units<KIND> units;
    Unit un;

    // The grid is the host's upper bound: clusters past the last unit leave.
    ptx::grid_dependency_wait();
    if (!units.get(pair, args, &un)) return;
    const uint64_t limit = wait_limit(args);
    // The weight gradient's stages are completed by both CTAs (the producers,
    // or the warps that clear a ragged end).  Walkers: both TMA warps, every
    // epilogue warp, the MMA warp, and the clearing warps or the asking warp.
    pair_setup(bar, GRAD ? 2 : 1, 2 + 16 + 1 + (GRAD ? 2 : 1), 8, &tmW, &tmA);

    const uint32_t tmem = bar->tmem_base;
    volatile int* abort = &bar->abort;
    bool failed = false;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        uint32_t stage = 0, phase = 0;
        int issued = 0;
        const bool issuer = ptx::elect_one_sync();
        const uint32_t full0 = ptx::map_to_cta(ptx::smem_addr(&bar->full[0]), 0);
        Asker asker;
        do {
            if (GRAD && leader && !asker.ask(bar, abort, limit)) {
                failed = true;
                break;
            }
            const int half = un.width / 2;                 // rows this CTA loads
            const int col0 = un.n0 + static_cast<int>(rank) * 128;
            const int first = un.row0 + static_cast<int>(rank) * half;
            // More than 64 rows come as one box (each load takes the warp time
            // that it does not have: six of them 650 clocks a K block).
            const bool whole = !GRAD && half > 64;
            const int boxes = GRAD ? half / 64 : (half + kBoxRows - 1) / kBoxRows;
            const uint32_t mine = static_cast<uint32_t>(
                kHalfBytes + (whole ? kHalfBytes : boxes * (GRAD ? kAtomBytes : kBoxRows * 128)));
            for (int b = 0; b < un.blocks; ++b) {
                if (!__all_sync(0xffffffffu,
                                ptx::mbar_wait(&bar->empty[stage], phase ^ 1u, abort, limit))) {
                    failed = true;
                    break;
                }
                const bool planted = pair == 0 && issued == args.drop_stage;
                if (!planted && issuer) {
                    uint8_t* w = base + stage * kStageBytes;
                    uint8_t* r = w + kHalfBytes;
                    const int kk = un.k0 + b * BK;
                    // A ragged end of the weight gradient lands on this CTA's
                    // own barrier of the stage first (one a stage: several
                    // ends can be in flight).
                    const bool ragged = GRAD && un.k1 - kk < BK;
                    uint32_t fb;
                    if (ragged) {
                        ptx::mbar_arrive_expect_tx(&bar->side_full[stage], mine);
                        fb = ptx::map_to_cta(ptx::smem_addr(&bar->side_full[stage]), rank);
                    } else {
                        fb = full0 + stage * 8;
                        if (leader) ptx::mbar_arrive_expect_tx(&bar->full[stage], 2 * mine);
                        else if (GRAD) ptx::mbar_arrive_remote(fb);
                    }
                    if constexpr (KIND == kWeight16KN) {
                        ptx::tma_load_3d_pair(w, &tmW, fb, col0, kk, un.group);
                        ptx::tma_load_3d_pair(w + kAtomBytes, &tmW, fb, col0 + 64, kk, un.group);
                    } else if constexpr (GRAD) {
                        ptx::tma_load_3d_pair(w, &tmW, fb, col0, kk, 0);
                        ptx::tma_load_3d_pair(w + kAtomBytes, &tmW, fb, col0 + 64, kk, 0);
                    } else {
                        ptx::tma_load_3d_pair(w, &tmW, fb, kk, col0, un.group);
                    }
                    if (whole) ptx::tma_load_3d_pair(r, &tmA128, fb, kk, first, 0);
                    for (int j = 0; j < (whole ? 0 : boxes); ++j) {
                        if constexpr (GRAD)
                            ptx::tma_load_3d_pair(r + j * kAtomBytes, &tmA, fb, first + j * 64, kk, 0);
                        else
                            ptx::tma_load_3d_pair(r + j * kBoxRows * 128, &tmA, fb, kk,
                                                  first + j * kBoxRows, 0);
                    }
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
        const uint32_t sW = ptx::smem_addr(base), sA = sW + kHalfBytes;
        constexpr bool WMN = KIND == kWeight16KN || GRAD;
        const uint64_t w0 = WMN ? ptx::smem_desc_sw128(sW, kAtomBytes, 1024)
                                : ptx::smem_desc_sw128(sW, 16, 1024);
        const uint64_t a0 = GRAD ? ptx::smem_desc_sw128(sA, kAtomBytes, 1024)
                                 : ptx::smem_desc_sw128(sA, 16, 1024);
        constexpr int WSTEP = (WMN ? 2048 : 32) >> 4, ASTEP = (GRAD ? 2048 : 32) >> 4;
        const bool issuer = ptx::elect_one_sync();
        do {
            // (No K blocks: an empty group's gradient.)
            const uint32_t idesc = args.idesc | static_cast<uint32_t>(un.width >> 3) << 17;
            for (int b = 0; b < un.blocks; ++b) {
                bool ok = true;
                if (b == 0) ok = ptx::mbar_wait(&bar->acc_empty[acc], acc_phase ^ 1u, abort, limit);
                ok = ok && ptx::mbar_wait(&bar->full[stage], phase, abort, limit);
                if (!__all_sync(0xffffffffu, ok)) {
                    failed = true;
                    break;
                }
                ptx::tc_fence_after();
                if (issuer) {
                    const uint64_t at = (stage * kStageBytes) >> 4;
                    const uint32_t d = tmem + acc * kMaxWidth;
                    if constexpr (GRAD) {
                        const int steps = min(4, (un.k1 - un.k0 - b * BK + 15) / 16);
                        for (int kk = 0; kk < steps; ++kk)
                            ptx::mma_f16<2>(d, w0 + at + kk * WSTEP, a0 + at + kk * ASTEP, idesc,
                                            b != 0 || kk != 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_f16<2>(d, w0 + at + kk * WSTEP, a0 + at + kk * ASTEP, idesc,
                                            b != 0 || kk != 0);
                    }
                    ptx::mma_commit<2>(&bar->empty[stage]);
                    if (b == un.blocks - 1) ptx::mma_commit<2>(&bar->acc_full[acc]);
                }
                __syncwarp();
                if (++stage == kStages) { stage = 0; phase ^= 1u; }
                if (b == un.blocks - 1) {
                    acc ^= 1u;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
        } while (!failed && walk.next(bar, abort, limit, &failed) &&
                 units.get(walk.unit, args, &un));
        if (failed && lane == 0) raise_error(args.err, abort, kErrMma);
        if (issuer) {
            ptx::mma_commit_local<2>(&bar->drain);
            ptx::mbar_wait(&bar->drain, 0, nullptr, limit);
        }
        __syncwarp();
    } else if (!GRAD && warp == 3 && leader) {
        // ---------------- the next units ----------------
        // (Asking takes the TMA warp 1200 clocks a unit, which the products' loads
        // do not have: 95 us for the products above, 88 without it.  The weight
        // gradient asks there, which measured better: 90 against 94.)
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
    } else if (GRAD && warp == 2) {
        // ---------------- ragged ends: clear the rows past the group's ----------------
        int issued = 0;
        uint32_t phases = 0;                               // a bit per stage
        do {
            issued += un.blocks;
            const int here = (un.k1 - un.k0) % BK;
            if (here == 0) continue;
            const int stage = (issued - 1) % kStages;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->side_full[stage], phases >> stage & 1u,
                                                        abort, limit))) {
                failed = true;
                break;
            }
            phases ^= 1u << stage;
            const uint32_t at = ptx::smem_addr(base) + stage * kStageBytes;
            // Only the MMA's last 16-row step reaches past `here`; its rows
            // are whole 128-byte lines of every 64-column atom (the swizzle
            // stays inside a line).
            const int pieces = ((here + 15) / 16 * 16 - here) * 8;
            const int atoms = 2 + un.width / 128;
            for (int j = 0; j < atoms; ++j)
                for (int p = lane; p < pieces; p += 32)
                    ptx::st_shared_v4(at + j * kAtomBytes + here * 128 + p * 16, 0, 0, 0, 0);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive_cluster(ptx::map_to_cta(ptx::smem_addr(&bar->full[stage]), 0));
        } while (walk.next(bar, abort, limit, &failed) && units.get(walk.unit, args, &un));
        if (failed && lane == 0) raise_error(args.err, abort, kErrProducer);
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        const int quarter = warp & 3, set = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* box = staging + (warp - 4) * kBoxBytes;
        const bool f16 = args.c_dtype == TILES_F16;
        // One chunk of 32 columns of this warp's 32 lanes leaves: v0 holds
        // lanes 0-15, v1 lanes 16-31, in the fragment layout.
        auto emit = [&](const uint32_t (&v0)[16], const uint32_t (&v1)[16], int col) {
            const int f0 = un.n0 + static_cast<int>(rank) * 128 + quarter * 32;
            const int row0 = un.row0 + col;
            const int64_t out0 = (GRAD ? static_cast<int64_t>(un.group) * args.stride_c : 0) +
                                 static_cast<int64_t>(row0) * args.ldc + f0;
            const int rows = un.end - row0, cols = args.n - f0;    // what is left to write
            if (rows <= 0 || cols <= 0) return;
            if (args.c_dtype == TILES_F32) {
                // Eight lanes write 32 consecutive bytes of a row.
                float* c = static_cast<float*>(args.c) + out0;
                const int f = lane >> 2;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = i * 8 + (lane & 3) * 2 + j;
                        if (r < rows) {
                            float* at = c + r * args.ldc + f;
                            if (f < cols) at[0] = __uint_as_float(v0[4 * i + j]);
                            if (f + 8 < cols) at[8] = __uint_as_float(v0[4 * i + 2 + j]);
                            if (f + 16 < cols) at[16] = __uint_as_float(v1[4 * i + j]);
                            if (f + 24 < cols) at[24] = __uint_as_float(v1[4 * i + 2 + j]);
                        }
                    }
                return;
            }
            box_begin();
            // Matrix q of a store is lanes 8q .. 8q+7; lane t addresses row
            // t%8 of matrix t/8.
            const uint32_t to = ptx::smem_addr(box);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ptx::st_matrix_x4_trans(to + box_piece(i * 8 + (lane & 7), lane >> 3),
                                        pack16(v0[4 * i], v0[4 * i + 1], f16),
                                        pack16(v0[4 * i + 2], v0[4 * i + 3], f16),
                                        pack16(v1[4 * i], v1[4 * i + 1], f16),
                                        pack16(v1[4 * i + 2], v1[4 * i + 3], f16));
            box_end(&tmC, args.tma_store, box, f0, row0, GRAD ? un.group : 0,
                    static_cast<uint16_t*>(args.c) + out0, args.ldc, rows, cols, GRAD);
        };
        uint32_t acc = 0, acc_phase = 0;
        do {
            uint32_t v0[16], v1[16];
            if (GRAD && un.blocks == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = v1[i] = 0;
                for (int col = set * 32; col < un.width; col += 64) emit(v0, v1, col);
                continue;
            }
            if (!__all_sync(0xffffffffu,
                            ptx::mbar_wait(&bar->acc_full[acc], acc_phase, abort, limit))) {
                failed = true;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t t = tmem + lanes + acc * kMaxWidth;
            for (int col = set * 32; col < un.width; col += 64) {
                ptx::tmem_ld_16x32(t + col, v0);
                ptx::tmem_ld_16x32(t + col + (16u << 16), v1);
                ptx::tmem_ld_wait();
                emit(v0, v1, col);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) hand_back(&bar->acc_empty[acc], leader);
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        } while (walk.next(bar, abort, limit, &failed) && units.get(walk.unit, args, &un));
        if (failed && lane == 0) raise_error(args.err, abort, kErrEpilogue);
        box_begin();                                       // the last box has been read
    }
    pair_teardown(tmem);
}

template <int KIND>
int launch_kind(const CUtensorMap& w, const CUtensorMap& a, const CUtensorMap& a128,
                const CUtensorMap& c, const ProductArgs& args, int units, cudaStream_t st) {
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(pair_kernel<KIND>, kSmemBytes, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    return launch_cluster(pair_kernel<KIND>, 2, dim3(static_cast<unsigned>(2 * units)),
                          dim3(kThreads), kSmemBytes, st, w, a, a128, c, args);
}

}  // namespace

int launch_pair(int kind, const CUtensorMap& weight, const CUtensorMap& rows,
                const CUtensorMap& rows128, const CUtensorMap& out, const ProductArgs& args,
                int units, cudaStream_t st) {
    switch (kind) {
        case kWeight16KN:
            return launch_kind<kWeight16KN>(weight, rows, rows128, out, args, units, st);
        case kWeight16NK:
            return launch_kind<kWeight16NK>(weight, rows, rows128, out, args, units, st);
        default: return launch_kind<kWeightGrad>(weight, rows, rows128, out, args, units, st);
    }
}

}  // namespace tiles

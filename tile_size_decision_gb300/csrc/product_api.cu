// C ABI of the dense 8-bit product, the grouped products and the grouped
// weight gradient (contracts in include/tiles.h): argument checks, tensor
// maps, the choice of a kernel and its launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "product_sm103a.cuh"

namespace tiles {
namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s per wait, as in the GEMM
constexpr int64_t kMaxSize = INT32_MAX / 2;

bool aligned(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int check_groups(int64_t groups, const int32_t* offsets) {
    if (groups < 1) return fail(TILES_ERR_INVALID_ARG, "groups must be >= 1");
    if (groups > kMaxGroups) return fail(TILES_ERR_TOO_LARGE, "more than %d groups", kMaxGroups);
    if (!offsets || !aligned(offsets, 4))
        return fail(TILES_ERR_INVALID_ARG, "offsets is null or not aligned to its element");
    return TILES_OK;
}

int check_workspace(const void* ws, size_t ws_bytes) {
    if (!ws || ws_bytes < static_cast<size_t>(kConvMinWorkspaceBytes))
        return fail(TILES_ERR_INVALID_ARG, "a workspace of at least %d bytes is required",
                    kConvMinWorkspaceBytes);
    if (!aligned(ws, 4)) return fail(TILES_ERR_MISALIGNED, "the workspace must be 4-byte aligned");
    return TILES_OK;
}

CUtensorMapDataType map_type(int dtype) {
    return dtype == TILES_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
           : dtype == TILES_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

int check_product(const tiles_product_desc* d, bool grouped) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    if (d->m < 0 || d->n < 1 || d->k < 1)
        return fail(TILES_ERR_INVALID_ARG, "m must be >= 0, n and k >= 1 (m=%lld n=%lld k=%lld)",
                    (long long)d->m, (long long)d->n, (long long)d->k);
    if (d->m > kMaxSize || d->n > kMaxSize || d->k > kMaxSize)
        return fail(TILES_ERR_TOO_LARGE, "a size exceeds 2^30");
    const bool fp8 = d->in_dtype == TILES_E4M3;
    if (!fp8 && (!grouped || (d->in_dtype != TILES_F16 && d->in_dtype != TILES_BF16)))
        return fail(TILES_ERR_UNSUPPORTED_DTYPE,
                    grouped ? "the operands must be f16, bf16 or e4m3" : "the operands must be e4m3");
    const int cb = dtype_bytes(d->out_dtype);
    if (!cb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "C must be f32, f16 or bf16");
    if (d->b_layout != TILES_B_KN && d->b_layout != TILES_B_NK)
        return fail(TILES_ERR_INVALID_ARG, "unknown weight layout %d", d->b_layout);
    if (fp8 && d->b_layout != TILES_B_NK)
        return fail(TILES_ERR_INVALID_ARG, "an e4m3 weight is stored n x k");
    if (grouped) {
        const int s = check_groups(d->groups, d->offsets);
        if (s != TILES_OK) return s;
    } else if (d->groups != 0) {
        return fail(TILES_ERR_INVALID_ARG, "a dense product has groups == 0");
    }
    if (d->m == 0) return TILES_OK;
    if (!d->a || !d->b || !d->c) return fail(TILES_ERR_INVALID_ARG, "null matrix pointer");
    if (fp8 && (!d->a_scales || !d->b_scales)) return fail(TILES_ERR_INVALID_ARG, "null scales");
    const int eb = fp8 ? 1 : 2;
    const int64_t brow = d->b_layout == TILES_B_KN ? d->n : d->k;
    const int64_t brows = d->b_layout == TILES_B_KN ? d->k : d->n;
    if (d->lda < d->k || d->ldb < brow || d->ldc < d->n)
        return fail(TILES_ERR_INVALID_ARG, "leading dimension smaller than the row length");
    if (grouped && d->groups > 1 && d->stride_b < (brows - 1) * d->ldb + brow)
        return fail(TILES_ERR_INVALID_ARG, "stride_b overlaps the weights");
    if (!aligned(d->a, 16) || !aligned(d->b, 16) || d->lda * eb % 16 || d->ldb * eb % 16 ||
        (grouped && d->groups > 1 && d->stride_b * eb % 16))
        return fail(TILES_ERR_MISALIGNED,
                    "a and b need 16-byte aligned bases, row pitches and group strides");
    if (!aligned(d->c, cb) || (fp8 && (!aligned(d->a_scales, 4) || !aligned(d->b_scales, 4))))
        return fail(TILES_ERR_MISALIGNED, "C or the scales are not aligned to their element");
    return TILES_OK;
}

// CTA pairs resident at once, asked of the runtime once per device.
int resident_pairs(int sms, int* pairs) {
    static std::atomic<int> known[64];
    int d = 0;
    const cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return fail(TILES_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    int n = d < 64 ? known[d].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        n = pair_max_groups(sms);
        if (d < 64) known[d].store(n, std::memory_order_relaxed);
    }
    *pairs = n;
    return TILES_OK;
}

// How a product runs: on CTA pairs, or with the few-rows kernel; the rows and
// columns of a tile, and the CTAs along K.
struct Choice { bool pair; int rows, cols, split; };

// The cheapest by a model in nanoseconds: a start, then the larger of
//   - the rounds over the resident blocks x (a round's own start and end + its
//     K blocks x the time of one), and
//   - the bytes at the measured copy rate, times how far a kernel stays from it.
// Few rows (two blocks an SM): a second resident block and the addition over a
// cluster cost extra.  8-bit pairs: a K block's time depends on the kernel
// (tiles up to 128 or 256 wide), not on the tile's width.  The constants are fitted
// to the times of 150 products on a GB300 with every kernel (m 1 to 25,000, n
// and k 128 to 4096, up to 32 groups): within 5 to 9% of them on average, and
// the choice within 1% of the best.  Both sides, in 8 bits: 16 rows of 4096 x
// 4096 5.4 us against 20.3 on pairs, 1000 x 4096 x 128 10.0 against 6.4; 32
// groups of 53 rows, 128 x 2816 in 16 bits, 16.6 against 11.8, 8 of 62 rows,
// 128 x 1024, 3.9 against 5.5.  Tiles of 128 rows never won: 8-bit sums of 128
// rows leave room for one block an SM.
Choice choose(int kind, int64_t m, int64_t n, int64_t k, int64_t groups, int sms, int pairs) {
    const bool fp8 = kind == kWeight8NK;
    const int64_t kb = (k + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
    // Row tiles: grouped, half a tile a group more than the rows fill, at
    // least one for every group that can have rows.
    auto row_tiles = [&](int64_t rows) {
        if (groups == 0) return (m + rows - 1) / rows;
        return std::max(std::min(groups, m), m / rows + groups / 2);
    };
    const int64_t eb = fp8 ? 1 : 2;
    const int64_t weights = groups == 0 ? 1 : std::min(groups, m);
    const double dram_ns = static_cast<double>((weights * n * k + m * k) * eb + 2 * m * n) / 6786.0;
    Choice best{};
    double best_ns = 0;
    auto offer = [&](const Choice& c, double ns) {
        if (best_ns == 0 || ns < best_ns) { best = c; best_ns = ns; }
    };
    struct Few { int rows; double start, round, block, second, cluster, far; };
    static constexpr Few few16[] = {{16, 1150, 2260, 250, 640, 35, 1.08},
                                    {32, 1000, 2720, 265, 900, 16, 1.10},
                                    {64, 570, 3710, 340, 1490, 5, 1.15}};
    static constexpr Few few8[] = {{16, 820, 2230, 310, 610, 35, 1.00},
                                   {32, 720, 2780, 360, 870, 8, 1.10},
                                   {64, 120, 4010, 465, 1760, 4, 1.20}};
    for (const Few& f : fp8 ? few8 : few16) {
        const int64_t units = row_tiles(f.rows) * ((n + 127) / 128);
        // CTAs along K: while the units leave SMs without a block, at least
        // two K blocks a CTA.
        int split = 1;
        while (split < 8 && units * split < sms && kb >= split * 4) split *= 2;
        const double rounds = static_cast<double>((units * split + 2 * sms - 1) / (2 * sms));
        const double work = rounds * (f.round + static_cast<double>((kb + split - 1) / split) * f.block) +
                            (units * split > sms ? f.second : 0);
        offer(Choice{false, f.rows, 128, split},
              f.start + std::max(work, dram_ns * f.far) + (split > 1 ? f.cluster * f.rows : 0));
    }
    // Pairs: 8-bit tiles as narrow as the rounds allow, in either kernel.
    struct Pair { int most, least; double start, round, block; };
    static constexpr Pair pair16[] = {{256, 256, 4400, 1350, 250}};
    static constexpr Pair pair8[] = {{256, 160, 3970, 1620, 460}, {128, 64, 3500, 1100, 300}};
    for (int i = 0; i < (fp8 ? 2 : 1); ++i) {
        const Pair& p = fp8 ? pair8[i] : pair16[i];
        int64_t fewest = INT64_MAX;
        int cols = p.most;
        for (int c = p.most; c >= p.least; c -= 32) {
            const int64_t rounds = (row_tiles(256) * ((n + c - 1) / c) + pairs - 1) / pairs;
            if (rounds <= fewest) { fewest = rounds; cols = c; }
        }
        offer(Choice{true, 256, cols, 1},
              p.start + std::max(static_cast<double>(fewest) * (p.round + kb * p.block),
                                 dram_ns * 1.05));
    }
    return best;
}

int run_product(const tiles_product_desc* d, bool grouped, void* ws, size_t ws_bytes, void* stream) {
    int s = check_product(d, grouped);
    if (s != TILES_OK) return s;
    if ((s = check_workspace(ws, ws_bytes)) != TILES_OK) return s;
    if (d->m == 0) return TILES_OK;
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    const bool fp8 = d->in_dtype == TILES_E4M3;
    const int kind = fp8 ? kWeight8NK : d->b_layout == TILES_B_NK ? kWeight16NK : kWeight16KN;
    const int eb = fp8 ? 1 : 2, bk = fp8 ? 128 : 64;
    const int64_t groups = grouped ? d->groups : 1;

    ProductArgs args{};
    args.m = static_cast<int32_t>(d->m);
    args.n = static_cast<int32_t>(d->n);
    args.k = static_cast<int32_t>(d->k);
    args.groups = grouped ? static_cast<int32_t>(d->groups) : 0;
    args.offsets = d->offsets;
    args.c = d->c;
    args.ldc = d->ldc;
    args.c_dtype = d->out_dtype;
    args.sa = d->a_scales;
    args.sb = d->b_scales;
    args.sa_row = d->a_scale_row;
    args.sa_block = d->a_scale_block;
    args.sb_row = d->b_scale_row;
    args.sb_block = d->b_scale_block;
    args.sb_group = grouped ? d->b_scale_group : 0;
    args.err = static_cast<int32_t*>(ws);
    args.wait_limit_ns = kWaitLimitNs;
    const PlantedFault planted = take_planted_fault();
    args.drop_stage = planted.stage;
    if (planted.stage >= 0) args.wait_limit_ns = planted.limit_ns;

    int pairs = 0;
    if ((s = resident_pairs(sms, &pairs)) != TILES_OK) return s;
    const Choice choice = choose(kind, d->m, d->n, d->k, grouped ? d->groups : 0, sms, pairs);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const char* what = grouped ? "grouped product" : "8-bit product";
    const bool kn = kind == kWeight16KN;
    const int64_t stride_b = groups > 1 ? d->stride_b : d->ldb;
    args.k_blocks = static_cast<int32_t>((d->k + bk - 1) / bk);
    args.n_blocks = static_cast<int32_t>((d->n + choice.cols - 1) / choice.cols);
    // Row tiles: exact when dense; grouped, every group may end inside one.
    const int64_t row_tiles = grouped ? d->m / choice.rows + std::min(groups, d->m)
                                      : (d->m + choice.rows - 1) / choice.rows;
    const int64_t units = row_tiles * args.n_blocks;
    if (units > INT32_MAX / 16) return fail(TILES_ERR_TOO_LARGE, "too many output tiles");
    // Boxes: one operand of a stage (MN-major: 64-column atoms).  In pairs half a
    // tile's columns (8 bits), and rows by 128 or, as a tile ends anywhere, by 32.
    const bool pair = choice.pair;
    CUtensorMap tw, ta;
    s = encode_box(&tw, map_type(d->in_dtype), d->b, kn ? d->n : d->k, kn ? d->k : d->n, groups,
                   d->ldb * eb, stride_b * eb, kn ? 64 : bk, kn ? 64 : pair && fp8 ? choice.cols / 2 : 128);
    if (s != TILES_OK) return s;
    s = encode_box(&ta, map_type(d->in_dtype), d->a, d->k, d->m, 1, d->lda * eb, d->lda * eb, bk,
                   !pair ? choice.rows : fp8 ? 128 : 32);
    if (s != TILES_OK) return s;
    const int mma_rows = pair ? 256 : 128, mma_cols = pair ? 0 : choice.rows;
    args.idesc = fp8 ? ptx::idesc_e4m3_f32acc(mma_rows, mma_cols)
                     : ptx::idesc_f16_f32acc_majors(d->in_dtype == TILES_BF16, kn, false, mma_rows,
                                                    mma_cols);
    if (!pair) {
        args.split = choice.split;
        return launch_status(launch_stream(kind, choice.rows, tw, ta, args, units, st), what);
    }
    args.tile_cols = choice.cols;
    CUtensorMap tc{};
    args.tma_store = encode_out_boxes(&tc, d->out_dtype, d->c, d->n, d->m, 1, d->ldc, d->ldc);
    if (fp8)
        return launch_status(launch_pair8(tw, ta, tc, args, static_cast<int>(units), st), what);
    CUtensorMap ta128;
    s = encode_box(&ta128, map_type(d->in_dtype), d->a, d->k, d->m, 1, d->lda * eb, d->lda * eb, bk,
                   128);
    if (s != TILES_OK) return s;
    return launch_status(launch_pair(kind, tw, ta, ta128, tc, args, static_cast<int>(units), st), what);
}

}  // namespace
}  // namespace tiles

using namespace tiles;

extern "C" {

int tiles_gemm_fp8(const tiles_product_desc* desc, void* ws, size_t ws_bytes, void* stream) {
    return run_product(desc, false, ws, ws_bytes, stream);
}

int tiles_grouped_gemm(const tiles_product_desc* desc, void* ws, size_t ws_bytes, void* stream) {
    return run_product(desc, true, ws, ws_bytes, stream);
}

int tiles_grouped_wgrad(const tiles_wgrad_desc* d, void* ws, size_t ws_bytes, void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    if (d->m < 0 || d->n < 1 || d->k < 1)
        return fail(TILES_ERR_INVALID_ARG, "m must be >= 0, n and k >= 1 (m=%lld n=%lld k=%lld)",
                    (long long)d->m, (long long)d->n, (long long)d->k);
    if (d->m > kMaxSize || d->n > kMaxSize || d->k > kMaxSize)
        return fail(TILES_ERR_TOO_LARGE, "a size exceeds 2^30");
    if (d->in_dtype != TILES_F16 && d->in_dtype != TILES_BF16)
        return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the operands must be f16 or bf16");
    const int ob = dtype_bytes(d->out_dtype);
    if (!ob) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "dw must be f32, f16 or bf16");
    int s = check_groups(d->groups, d->offsets);
    if (s != TILES_OK) return s;
    if (!d->dw || (d->m > 0 && (!d->a || !d->dc)))
        return fail(TILES_ERR_INVALID_ARG, "null matrix pointer");
    if (d->lda < d->k || d->lddc < d->n || d->lddw < d->n)
        return fail(TILES_ERR_INVALID_ARG, "leading dimension smaller than the row length");
    if (d->groups > 1 && d->stride_dw < (d->k - 1) * d->lddw + d->n)
        return fail(TILES_ERR_INVALID_ARG, "stride_dw overlaps the gradients");
    if ((d->m > 0 && (!aligned(d->a, 16) || !aligned(d->dc, 16))) || d->lda % 8 || d->lddc % 8)
        return fail(TILES_ERR_MISALIGNED, "a and dc need 16-byte aligned bases and row pitches");
    if (!aligned(d->dw, ob)) return fail(TILES_ERR_MISALIGNED, "dw is not aligned to its element");
    if (d->groups * ((d->k + 127) / 128) > INT32_MAX / ((d->n + 127) / 128))
        return fail(TILES_ERR_TOO_LARGE, "too many output tiles");
    if ((s = check_workspace(ws, ws_bytes)) != TILES_OK) return s;
    // The tile of the products with other names: dc is the weight side, the
    // columns of a are the rows, and the group's rows the contraction.
    ProductArgs args{};
    args.m = static_cast<int32_t>(d->m);
    args.n = static_cast<int32_t>(d->n);
    args.k = static_cast<int32_t>(d->k);
    args.groups = static_cast<int32_t>(d->groups);
    args.offsets = d->offsets;
    args.n_blocks = static_cast<int32_t>((d->n + 255) / 256);
    args.c = d->dw;
    args.ldc = d->lddw;
    args.stride_c = d->stride_dw;
    args.c_dtype = d->out_dtype;
    args.idesc = ptx::idesc_f16_f32acc_majors(d->in_dtype == TILES_BF16, true, true, 256, 0);
    args.err = static_cast<int32_t*>(ws);
    args.wait_limit_ns = kWaitLimitNs;
    const PlantedFault planted = take_planted_fault();
    args.drop_stage = planted.stage;
    if (planted.stage >= 0) args.wait_limit_ns = planted.limit_ns;
    // No rows: every group is empty and nothing is loaded; the maps then
    // only have to be valid.
    const bool none = d->m == 0;
    alignas(16) static const char nothing[16] = {};
    CUtensorMap tw, ta;
    s = encode_box(&tw, map_type(d->in_dtype), none ? nothing : d->dc, d->n, none ? 1 : d->m, 1,
                   d->lddc * 2, d->lddc * 2, 64, 64);
    if (s != TILES_OK) return s;
    s = encode_box(&ta, map_type(d->in_dtype), none ? nothing : d->a, d->k, none ? 1 : d->m, 1,
                   d->lda * 2, d->lda * 2, 64, 64);
    if (s != TILES_OK) return s;
    const int64_t units = d->groups * ((d->k + 255) / 256) * args.n_blocks;
    CUtensorMap tc{};
    args.tma_store = encode_out_boxes(&tc, d->out_dtype, d->dw, d->n, d->k, d->groups, d->lddw,
                                      d->groups > 1 ? d->stride_dw : d->lddw);
    return launch_status(launch_pair(kWeightGrad, tw, ta, ta, tc, args, static_cast<int>(units),
                                     static_cast<cudaStream_t>(stream)),
                         "grouped weight gradient");
}

}  // extern "C"

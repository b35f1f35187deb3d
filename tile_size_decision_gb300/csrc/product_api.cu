// C ABI of the dense 8-bit product, the grouped products and the grouped
// weight gradient (contracts in include/tiles.h): argument checks, tensor
// maps, the choice of a kernel and its launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "product_choice.h"
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
    const Choice choice = choose(fp8, d->m, d->n, d->k, grouped ? d->groups : 0, sms, pairs);
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

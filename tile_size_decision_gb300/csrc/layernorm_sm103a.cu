// Layer norm with the residual's addition (16-bit, fp32 or scaled 8-bit
// output) and its gradients.
//
// As the root-mean-square norm, both read and write every element once and
// compute a few operations per byte: DRAM bounds them.  The row's sums are
// taken twice from registers: first a mean m in fp32, then the sums of d = h - m
// and of d^2, which give what m was off by, c = mean(d), and the variance
// mean(d^2) - c^2.  So a row whose mean is far larger than its spread loses
// nothing (with c left out the error of m, 2^-24 |m|, would shift all of y).
#include "row_ops.cuh"

namespace tiles {
namespace {

struct LayerArgs {
    int64_t rows, cols;
    const void* x;
    const void* residual;
    const void* weight;
    const void* bias;
    void* h;
    void* y;
    float* scales;
    int64_t ldx, ldr, ldh, ldy, scale_row, scale_block;
    float eps;
    int32_t weight_dtype;
};

// (var + eps)^(-1/2) from the mean of d^2 and of d.  The variance is no less
// than 0, whatever the two roundings leave; a NaN stays one.
__device__ __forceinline__ float inverse_root(float square, float off, float eps) {
    const float var = square - off * off;
    return rsqrtf((var < 0.0f ? 0.0f : var) + eps);
}

// One row per blockDim.x threads, blockDim.y rows per block; the layout of
// vectors over threads is the root-mean-square norm's.  VPT == 0 takes rows of
// any length: it reads h again from x and the residual for the variance and
// for the output.
template <typename T, int VPT, bool VEC, bool FP8>
__global__ void __launch_bounds__(kMaxThreads)
    layernorm_kernel(const LayerArgs a) {
    __shared__ float slots[64 + 128];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;                    // whole warps: blockDim.y > 1 only with 32 threads a row
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.0f / static_cast<float>(cols);
    auto load_h = [&](int c, float (&v)[8]) {
        load8<T, VEC>(x, c, cols, v);
        if (r) {
            float q[8];
            load8<T, VEC>(r, c, cols, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
        }
    };
    // v - mean; columns past the row's end stay zero.
    auto centre = [&](int c, float (&v)[8], float mean) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = column<VEC>(c, i) < cols ? v[i] - mean : 0.0f;
    };
    auto emit = [&](int c, const float (&v)[8], float rstd) {
        float w[8], y[8];
        load8_any<VEC>(a.weight, a.weight_dtype, c, cols, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * rstd * w[i];
        if (a.bias) {
            load8_any<VEC>(a.bias, a.weight_dtype, c, cols, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += w[i];
        }
        if constexpr (FP8) {
            // Zeros past the row's end times rstd may be NaN; they must not
            // reach the short last block's scale.
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (column<VEC>(c, i) >= cols) y[i] = 0.0f;
            const float s = block_scale(block_amax(amax8(y))), inv = reciprocal(s);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= inv;
            store8_e4m3<VEC>(static_cast<uint8_t*>(a.y) + row * a.ldy, c, cols, y);
            if ((threadIdx.x & 15) == 0 && c < cols)
                a.scales[row * a.scale_row + c / kBlock * a.scale_block] = s;
        } else {
            store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy, c, cols, y);
        }
    };
    const int step = blockDim.x * 8;
    float sum[1] = {0.0f}, sq[2] = {0.0f, 0.0f};   // sum h; sums of d, d^2
    if constexpr (VPT > 0) {
        float v[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) load_h(j * step + threadIdx.x * 8, v[j]);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (h) store8<T, VEC>(h, j * step + threadIdx.x * 8, cols, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[j][i];
        }
        row_sum(sum, slots, 0);
        const float mean = sum[0] * inv_n;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            centre(j * step + threadIdx.x * 8, v[j], mean);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sq[0] += v[j][i];
                sq[1] += v[j][i] * v[j][i];
            }
        }
        row_sum(sq, slots + 64, 0);
        const float off = sq[0] * inv_n, rstd = inverse_root(sq[1] * inv_n, off, a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] -= off;
            emit(j * step + threadIdx.x * 8, v[j], rstd);
        }
    } else {
        for (int c0 = 0; c0 < cols; c0 += step) {
            float v[8];
            load_h(c0 + threadIdx.x * 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[i];
        }
        row_sum(sum, slots, 0);
        const float mean = sum[0] * inv_n;
        for (int c0 = 0; c0 < cols; c0 += step) {
            const int c = c0 + threadIdx.x * 8;
            float v[8];
            load_h(c, v);
            centre(c, v, mean);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sq[0] += v[i];
                sq[1] += v[i] * v[i];
            }
        }
        row_sum(sq, slots + 64, 0);
        const float off = sq[0] * inv_n, rstd = inverse_root(sq[1] * inv_n, off, a.eps);
        for (int c0 = 0; c0 < cols; c0 += step) {
            const int c = c0 + threadIdx.x * 8;
            float v[8];
            load_h(c, v);
            // h may be stored over x or the residual: after its own read.
            if (h) store8<T, VEC>(h, c, cols, v);
            centre(c, v, mean);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] -= off;
            emit(c, v, rstd);
        }
    }
}

struct LayerGradArgs {
    int64_t rows, cols;
    const void* dy;
    const void* h;
    const void* weight;
    const void* dh;
    void* dx;
    float* partials;       // [gridDim.x][2][cols]: of the weight, of the bias
    int64_t lddy, ldh, lddh, lddx;
    float eps;
    int32_t weight_dtype;
};

// Each block sweeps rows, gridDim.x * blockDim.y apart; a thread keeps the same
// columns throughout, so its parts of the weight's and the bias's gradient
// stay in registers until the block's one write to `partials` (rows short
// enough for one warp go eight to a block, whose parts are added first).
// blockIdx.y picks a span of columns when a row is longer than one block holds
// (a vector a thread): each span then reads the whole row for the sums and
// writes its own columns.
template <typename T, bool VEC, bool SPANS>
__global__ void __launch_bounds__(512)
    layernorm_grad_kernel(const LayerGradArgs a) {
    __shared__ float slots[64 + 256];
    extern __shared__ float side[];                // blockDim.y > 1: the other warps' parts
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int step = blockDim.x * 8;
    const int cols = static_cast<int>(a.cols);
    const int first = static_cast<int>(blockIdx.y) * step;
    const int c = first + threadIdx.x * 8;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    float dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * blockDim.y) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* h = static_cast<const T*>(a.h) + row * a.ldh;
        const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
        float g[8], v[8], w[8], past[8];
        load8<T, VEC>(dy, c, cols, g);
        load8<T, VEC>(h, c, cols, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) past[i] = 0.0f;
        if (VEC && dh) load8<T, VEC>(dh, c, cols, past);
        load8_any<VEC>(a.weight, a.weight_dtype, c, cols, w);
        float m[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) m[0] += v[i];
        if constexpr (SPANS) {
            for (int c0 = 0; c0 < cols; c0 += step) {
                if (c0 == first) continue;
                float q[8];
                load8<T, VEC>(h, c0 + threadIdx.x * 8, cols, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) m[0] += q[i];
            }
        }
        row_sum(m, slots, 0);
        const float mean = m[0] * inv_n;
        // Sums of d, d^2, g = dy w and g d; columns past the row's end have g = 0
        // and are kept out of d.
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = column<VEC>(c, i) < cols ? v[i] - mean : 0.0f;
            s[0] += v[i];
            s[1] += v[i] * v[i];
            s[2] += g[i] * w[i];
            s[3] += g[i] * w[i] * v[i];
        }
        if constexpr (SPANS) {
            for (int c0 = 0; c0 < cols; c0 += step) {
                if (c0 == first) continue;
                const int at = c0 + threadIdx.x * 8;
                float p[8], q[8], u[8];
                load8<T, VEC>(dy, at, cols, p);
                load8<T, VEC>(h, at, cols, q);
                load8_any<VEC>(a.weight, a.weight_dtype, at, cols, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = column<VEC>(at, i) < cols ? q[i] - mean : 0.0f;
                    s[0] += d;
                    s[1] += d * d;
                    s[2] += p[i] * u[i];
                    s[3] += p[i] * u[i] * d;
                }
            }
        }
        row_sum(s, slots + 64, 0);
        const float off = s[0] * inv_n, rstd = inverse_root(s[1] * inv_n, off, a.eps);
        const float level = s[2] * inv_n * rstd;
        const float back = (s[3] - off * s[2]) * inv_n * rstd * rstd * rstd;
        if (!VEC && dh) load8<T, VEC>(dh, c, cols, past);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] -= off;
            o[i] = g[i] * w[i] * rstd - level - v[i] * back + past[i];
            dw[i] += g[i] * v[i] * rstd;
            db[i] += g[i];
        }
        store8<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx, c, cols, o);
    }
    if (blockDim.y > 1) {                          // then blockDim.x == 32: one warp a row
        if (threadIdx.y > 0)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                side[(threadIdx.y - 1) * 512 + i * 32 + threadIdx.x] = dw[i];
                side[(threadIdx.y - 1) * 512 + 256 + i * 32 + threadIdx.x] = db[i];
            }
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] += side[y * 512 + i * 32 + threadIdx.x];
                db[i] += side[y * 512 + 256 + i * 32 + threadIdx.x];
            }
    }
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (column<VEC>(c, i) < cols) {
            out[column<VEC>(c, i)] = dw[i];
            out[a.cols + column<VEC>(c, i)] = db[i];
        }
}

template <typename T, bool VEC, bool FP8>
int launch_layer(const LayerArgs& a, cudaStream_t st) {
    const int64_t vectors = (a.cols + 7) / 8;
    // One vector a thread for as long as a block can hold the row: a row's loads
    // are then all in flight at once.
    int vpt = 1;
    while (vpt <= 4 && (vectors + vpt - 1) / vpt > kMaxThreads) vpt *= 2;
    if (vpt > 4)
        return launch(layernorm_kernel<T, 0, VEC, FP8>, dim3(static_cast<unsigned>(a.rows)),
                      dim3(kMaxThreads, 1), 0, st, a);
    const int threads = static_cast<int>(((vectors + vpt - 1) / vpt + 31) / 32 * 32);
    const int per_block = threads == 32 ? 8 : 1;
    const dim3 grid(static_cast<unsigned>((a.rows + per_block - 1) / per_block));
    const dim3 block(threads, per_block);
    switch (vpt) {
        case 1: return launch(layernorm_kernel<T, 1, VEC, FP8>, grid, block, 0, st, a);
        case 2: return launch(layernorm_kernel<T, 2, VEC, FP8>, grid, block, 0, st, a);
        default: return launch(layernorm_kernel<T, 4, VEC, FP8>, grid, block, 0, st, a);
    }
}

template <typename T>
int launch_layer_any(const LayerArgs& a, bool vec, bool fp8, cudaStream_t st) {
    if (vec) return fp8 ? launch_layer<T, true, true>(a, st) : launch_layer<T, true, false>(a, st);
    return fp8 ? launch_layer<T, false, true>(a, st) : launch_layer<T, false, false>(a, st);
}

struct LayerGradGeometry { int threads, per_block, blocks, spans; };

// The blocks that sweep the rows, each of which writes one partial.
LayerGradGeometry layer_grad_geometry(int64_t rows, int64_t cols, int sms) {
    LayerGradGeometry g;
    const int64_t vectors = (cols + 7) / 8;
    g.threads = static_cast<int>(std::min<int64_t>((vectors + 31) / 32 * 32, 512));
    g.spans = static_cast<int>((vectors + g.threads - 1) / g.threads);
    g.per_block = g.threads == 32 ? 8 : 1;
    const int64_t sweeps = (rows + g.per_block - 1) / g.per_block;
    const int per_sm = std::max(1, std::min(16, 1024 / (g.threads * g.per_block)));
    g.blocks = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(sweeps, static_cast<int64_t>(sms) * per_sm)));
    return g;
}

size_t layer_grad_bytes(int64_t rows, int64_t cols, int sms) {
    return kConvMinWorkspaceBytes + static_cast<size_t>(layer_grad_geometry(rows, cols, sms).blocks) *
                                        static_cast<size_t>(cols) * 8;
}

template <typename T>
int launch_layer_grad(const LayerGradArgs& a, bool vec, int sms, int* parts, cudaStream_t st) {
    const LayerGradGeometry g = layer_grad_geometry(a.rows, a.cols, sms);
    *parts = g.blocks;
    const dim3 grid(g.blocks, g.spans), block(g.threads, g.per_block);
    const size_t side = g.per_block > 1 ? (g.per_block - 1) * 512 * 4 : 0;
    if (g.spans > 1)
        return vec ? launch(layernorm_grad_kernel<T, true, true>, grid, block, side, st, a)
                   : launch(layernorm_grad_kernel<T, false, true>, grid, block, side, st, a);
    return vec ? launch(layernorm_grad_kernel<T, true, false>, grid, block, side, st, a)
               : launch(layernorm_grad_kernel<T, false, false>, grid, block, side, st, a);
}

}  // namespace
}  // namespace tiles

using namespace tiles;

extern "C" {

int tiles_layernorm(const tiles_layernorm_desc* d, void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_sizes(d->rows, d->cols);
    if (s != TILES_OK) return s;
    const int eb = dtype_bytes(d->dtype);
    const bool fp8 = d->out_dtype == TILES_E4M3;
    if (!eb || (!fp8 && d->out_dtype != d->dtype))
        return fail(TILES_ERR_UNSUPPORTED_DTYPE,
                    "x must be f16, bf16 or f32, and the output of its type or e4m3");
    if (d->rows == 0) return TILES_OK;
    if ((s = check_weight(d->weight, d->weight_dtype)) != TILES_OK) return s;
    if (!element_aligned(d->bias, dtype_bytes(d->weight_dtype)))
        return fail(TILES_ERR_MISALIGNED, "bias is not aligned to its element");
    if ((s = check_matrix("x", d->x, d->ldx, d->cols, eb)) != TILES_OK) return s;
    if (d->residual && (s = check_matrix("residual", d->residual, d->ldr, d->cols, eb)) != TILES_OK)
        return s;
    if (d->h && (s = check_matrix("h", d->h, d->ldh, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("y", d->y, d->ldy, d->cols, fp8 ? 1 : eb)) != TILES_OK) return s;
    if (fp8 && (!d->scales || !element_aligned(d->scales, 4)))
        return fail(TILES_ERR_INVALID_ARG, "an e4m3 output needs aligned scales");
    LayerArgs a{d->rows, d->cols, d->x, d->residual, d->weight, d->bias, d->h, d->y, d->scales,
                d->ldx, d->ldr, d->ldh, d->ldy, d->scale_row, d->scale_block, d->eps,
                d->weight_dtype};
    const bool vec = d->cols % 8 == 0 && whole16(d->x, d->ldx, eb) &&
                     whole16(d->residual, d->ldr, eb) && whole16(d->h, d->ldh, eb) &&
                     whole16(d->weight, 0, 1) && whole16(d->bias, 0, 1) &&
                     (fp8 ? whole8(d->y, d->ldy) : whole16(d->y, d->ldy, eb));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int e;
    if (d->dtype == TILES_BF16) e = launch_layer_any<__nv_bfloat16>(a, vec, fp8, st);
    else if (d->dtype == TILES_F16) e = launch_layer_any<__half>(a, vec, fp8, st);
    else e = launch_layer_any<float>(a, vec, fp8, st);
    return launch_status(e, "layer norm");
}

size_t tiles_layernorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    if (check_sizes(rows, cols) != TILES_OK) return 0;
    int sms = 0;
    if (current_sm_count(&sms) != TILES_OK) return 0;
    return layer_grad_bytes(rows, cols, sms);
}

int tiles_layernorm_grad(const tiles_layernorm_grad_desc* d, void* ws, size_t ws_bytes,
                         void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_sizes(d->rows, d->cols);
    if (s != TILES_OK) return s;
    const int eb = dtype_bytes(d->dtype);
    if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "dy, h and dx must be f16, bf16 or f32");
    if (!d->dweight || !element_aligned(d->dweight, 4) || !d->dbias || !element_aligned(d->dbias, 4))
        return fail(TILES_ERR_INVALID_ARG, "dweight or dbias is null or not aligned to its element");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d->rows == 0) {
        cudaError_t e = cudaMemsetAsync(d->dweight, 0, static_cast<size_t>(d->cols) * 4, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(d->dbias, 0, static_cast<size_t>(d->cols) * 4, st);
        return launch_status(e, "layer norm gradient");
    }
    if ((s = check_weight(d->weight, d->weight_dtype)) != TILES_OK) return s;
    if ((s = check_matrix("dy", d->dy, d->lddy, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("h", d->h, d->ldh, d->cols, eb)) != TILES_OK) return s;
    if (d->dh && (s = check_matrix("dh", d->dh, d->lddh, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("dx", d->dx, d->lddx, d->cols, eb)) != TILES_OK) return s;
    if (!ws) return fail(TILES_ERR_INVALID_ARG, "the layer norm gradient needs a workspace");
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(TILES_ERR_MISALIGNED, "the workspace must be 16-byte aligned");
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    const size_t need = layer_grad_bytes(d->rows, d->cols, sms);
    if (ws_bytes < need)
        return fail(TILES_ERR_INVALID_ARG, "the layer norm gradient needs %zu workspace bytes", need);
    LayerGradArgs a{d->rows, d->cols, d->dy, d->h, d->weight, d->dh, d->dx,
                    reinterpret_cast<float*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes),
                    d->lddy, d->ldh, d->lddh, d->lddx, d->eps, d->weight_dtype};
    const bool vec = d->cols % 8 == 0 && whole16(d->dy, d->lddy, eb) && whole16(d->h, d->ldh, eb) &&
                     whole16(d->dh, d->lddh, eb) && whole16(d->dx, d->lddx, eb) &&
                     whole16(d->weight, 0, 1);
    int e;
    int parts = 0;
    if (d->dtype == TILES_BF16) e = launch_layer_grad<__nv_bfloat16>(a, vec, sms, &parts, st);
    else if (d->dtype == TILES_F16) e = launch_layer_grad<__half>(a, vec, sms, &parts, st);
    else e = launch_layer_grad<float>(a, vec, sms, &parts, st);
    if (e != cudaSuccess) return launch_status(e, "layer norm gradient");
    e = launch_reduce_partials(a.partials, d->cols, parts, d->dweight, d->dbias, st);
    return launch_status(e, "layer norm gradient reduction");
}

}  // extern "C"

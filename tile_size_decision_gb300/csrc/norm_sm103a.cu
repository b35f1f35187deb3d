// Root-mean-square norm with the residual's addition (16-bit, fp32 or scaled
// 8-bit output), its gradients, and the block quantiser of 8-bit matrices.
//
// All three read and write every element once and compute a few operations
// per byte: DRAM bounds them.  A row's elements stay in registers between
// the reduction and the output, so nothing is read twice.
#include <algorithm>
#include <cfloat>

#include "row_ops.cuh"

namespace tiles {
namespace {

// The shortcut of the kernel for many long rows (h * weight first) holds from
// this magnitude of h * weight on, and for zeros of rows that are not quieter
// than this 1 / rms: there even what fp32 lost below 2^-149 rounds to zero in 8
// bits.
constexpr float kQuiet = 0x1p-100f, kZeroRstd = 0x1p13f;

struct NormArgs {
    int64_t rows, cols;
    const void* x;
    const void* residual;
    const void* weight;
    void* h;
    void* y;
    float* scales;
    int64_t ldx, ldr, ldh, ldy, scale_row, scale_block;
    float eps;
    int32_t weight_dtype;
};

// One row per blockDim.x threads, blockDim.y rows per block.  Thread t holds
// the row's 8-element vectors t, t + blockDim.x, ... (VPT of them), so 16
// neighbouring lanes hold one block of 128 columns.  VPT == 0 takes rows of
// any length: it computes h again from x and the residual for the output.
template <typename T, int VPT, bool VEC, bool FP8>
__global__ void __launch_bounds__(kMaxThreads)
    rmsnorm_kernel(const NormArgs a) {
    __shared__ float slots[64];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;                    // whole warps: blockDim.y > 1 only with 32 threads a row
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
    const int cols = static_cast<int>(a.cols);
    auto load_h = [&](int c, float (&v)[8]) {
        load8<T, VEC>(x, c, cols, v);
        if (r) {
            float q[8];
            load8<T, VEC>(r, c, cols, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
        }
    };
    auto emit = [&](int c, const float (&v)[8], float rstd) {
        float w[8], y[8];
        load8_any<VEC>(a.weight, a.weight_dtype, c, cols, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * rstd * w[i];
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
    float sum[1] = {0.0f};
    if constexpr (VPT > 0) {
        float v[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) load_h(j * step + threadIdx.x * 8, v[j]);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (h) store8<T, VEC>(h, j * step + threadIdx.x * 8, cols, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[j][i] * v[j][i];
        }
        row_sum(sum, slots, 0);
        const float rstd = rsqrtf(sum[0] / static_cast<float>(a.cols) + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) emit(j * step + threadIdx.x * 8, v[j], rstd);
    } else {
        for (int c0 = 0; c0 < cols; c0 += step) {
            float v[8];
            load_h(c0 + threadIdx.x * 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[i] * v[i];
        }
        row_sum(sum, slots, 0);
        const float rstd = rsqrtf(sum[0] / static_cast<float>(a.cols) + a.eps);
        for (int c0 = 0; c0 < cols; c0 += step) {
            float v[8];
            load_h(c0 + threadIdx.x * 8, v);
            // h may be stored over x or the residual: after its own read.
            if (h) store8<T, VEC>(h, c0 + threadIdx.x * 8, cols, v);
            emit(c0 + threadIdx.x * 8, v, rstd);
        }
    }
}

// The same with the rows' pieces 16-byte aligned: the block takes rows
// blockIdx.x, + gridDim.x, ..., the next two of them on their way in while one
// is worked on.  DRAM bounds it: 16384 x 4096 bf16 rows with a residual, to
// e4m3, 72.6 us, 95% of the measured copy bandwidth; without a residual the
// work per byte does (11127 x 2728, 25.9 us, 53%; 25.1 without the check for
// blocks that take the definition's order).
template <typename T, int VPT, bool FP8, bool RES>
__global__ void __launch_bounds__(kRingThreads)
    rmsnorm_ring_kernel(const NormArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[64];
    const int threads = blockDim.x;
    RowRing<T, RES ? 2 : 1, VPT> ring{ring_smem + threadIdx.x};
    const int step = blockDim.x * 8, tid = threadIdx.x, cols = static_cast<int>(a.cols);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = gridDim.x, row0 = blockIdx.x;
    auto fetch = [&](int64_t row, int slot) {
        if (row < a.rows) {
            ring.copy(slot, 0, static_cast<const T*>(a.x) + row * a.ldx, step, tid, threads, cols);
            if constexpr (RES)
                ring.copy(slot, 1, static_cast<const T*>(a.residual) + row * a.ldr, step, tid, threads,
                          cols);
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(row0 + i * stride, i);
    float w[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        load8_any<true>(a.weight, a.weight_dtype, j * step + tid * 8, cols, w[j]);
    const float inv_n = 1.0f / static_cast<float>(cols);
    int slot = 0, turn = 0;
    for (int64_t row = row0; row < a.rows; row += stride, turn ^= 1) {
        const int refill = slot == 0 ? kRing - 1 : slot - 1;
        fetch(row + (kRing - 1) * stride, refill);
        ptx::cp_async_wait_groups<kRing - 1>();
        // What does not need the norm comes before the row's sum: h leaves and,
        // on the way to 8 bits, h becomes h * weight, and the blocks'
        // magnitudes are taken of that.  (16-bit results take h / rms first:
        // h * weight may be out of fp32's range where y is not.)
        float v[VPT][8], amax[VPT], sum[1] = {0.0f};
        auto read_h = [&](int j, float (&h)[8]) {
            const bool in = j * step + tid * 8 < cols;
            ring.read(slot, 0, j, in, threads, h);
            if constexpr (RES) {
                float q[8];
                ring.read(slot, 1, j, in, threads, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] += q[i];
            }
        };
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * step + tid * 8;
            read_h(j, v[j]);
            if (a.h) store8<T, true>(static_cast<T*>(a.h) + row * a.ldh, c, cols, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] += v[j][i] * v[j][i];
                if constexpr (FP8) v[j][i] *= w[j][i];
            }
            if constexpr (FP8) amax[j] = block_amax(amax8(v[j]));
        }
        row_sum(sum, slots, turn);
        const float rstd = rsqrtf(sum[0] * inv_n + a.eps);
        bool again = false;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * step + tid * 8;
            if constexpr (FP8) {
                const float s = block_scale(amax[j] * rstd);
                // (The bound is for a block of zeros in a quiet row.)
                const float factor = min_nan(rstd * reciprocal(s), FLT_MAX);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= factor;
                again |= !(amax[j] >= kQuiet && amax[j] <= FLT_MAX) &&
                         !(amax[j] == 0.0f && rstd <= kZeroRstd);
                store8_e4m3<true>(static_cast<uint8_t*>(a.y) + row * a.ldy, c, cols, v[j]);
                if ((tid & 15) == 0 && c < cols)
                    a.scales[row * a.scale_row + c / kBlock * a.scale_block] = s;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * w[j][i];
                store8<T, true>(static_cast<T*>(a.y) + row * a.ldy, c, cols, v[j]);
            }
        }
        // Where a block's h * weight left fp32's range, or is so quiet that it
        // may have, the warp's blocks once more, as they are defined.
        if (FP8 && __any_sync(0xffffffffu, again)) {
#pragma unroll 1
            for (int j = 0; j < VPT; ++j) {
                const int c = j * step + tid * 8;
                float y[8], u[8];
                read_h(j, y);
                load8_any<true>(a.weight, a.weight_dtype, c, cols, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = c < cols ? y[i] * rstd * u[i] : 0.0f;
                const float s = block_scale(block_amax(amax8(y))), inv = reciprocal(s);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= inv;
                store8_e4m3<true>(static_cast<uint8_t*>(a.y) + row * a.ldy, c, cols, y);
                if ((tid & 15) == 0 && c < cols)
                    a.scales[row * a.scale_row + c / kBlock * a.scale_block] = s;
            }
        }
        if (++slot == kRing) slot = 0;
    }
}

struct GradArgs {
    int64_t rows, cols;
    const void* dy;
    const void* h;
    const void* weight;
    const void* dh;
    void* dx;
    float* partials;       // [gridDim.x][cols]
    int64_t lddy, ldh, lddh, lddx;
    float eps;
    int32_t weight_dtype;
};

// Each block sweeps rows, gridDim.x * blockDim.y apart; a thread keeps the same
// columns throughout, so its part of the weight gradient stays in registers
// until the block's one write to `partials` (rows short enough for one warp
// go eight to a block, whose parts are added first).  blockIdx.y picks a span of
// columns when a row is longer than one block holds (a vector a thread): each
// span then reads the whole row for the two sums and writes its own columns.
template <typename T, bool VEC, bool SPANS>
__global__ void __launch_bounds__(512, 2)
    rmsnorm_grad_kernel(const GradArgs a) {
    __shared__ float slots[128];
    extern __shared__ float side[];                // blockDim.y > 1: the other warps' parts
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int step = blockDim.x * 8;
    const int cols = static_cast<int>(a.cols);
    const int first = static_cast<int>(blockIdx.y) * step;
    const int c = first + threadIdx.x * 8;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    float dw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.0f;
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * blockDim.y, turn ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* h = static_cast<const T*>(a.h) + row * a.ldh;
        const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
        float g[8], v[8], w[8], past[8];
        load8<T, VEC>(dy, c, cols, g);
        load8<T, VEC>(h, c, cols, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) past[i] = 0.0f;
        // dh with the others where it is one load (8192 x 4096 fp32: 88 us
        // against 95), after the sums where it is eight (3000 x 3001: 40
        // against 45: these instances spill 48 to 80 bytes a thread as it is).
        if (VEC && dh) load8<T, VEC>(dh, c, cols, past);
        load8_any<VEC>(a.weight, a.weight_dtype, c, cols, w);
        float s[2] = {0.0f, 0.0f};                 // sum h^2, sum dy w h
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[0] += v[i] * v[i];
            s[1] += g[i] * w[i] * v[i];
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
                    s[0] += q[i] * q[i];
                    s[1] += p[i] * u[i] * q[i];
                }
            }
        }
        row_sum(s, slots, turn);
        const float rstd = rsqrtf(s[0] * inv_n + a.eps);
        const float back = s[1] * inv_n * rstd * rstd * rstd;
        if (!VEC && dh) load8<T, VEC>(dh, c, cols, past);
        load8_any<VEC>(a.weight, a.weight_dtype, c, cols, w);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = g[i] * w[i] * rstd - v[i] * back + past[i];
            dw[i] += g[i] * v[i] * rstd;
        }
        store8<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx, c, cols, o);
    }
    if (blockDim.y > 1) {                          // then blockDim.x == 32: one warp a row
        if (threadIdx.y > 0)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                side[(threadIdx.y - 1) * 256 + i * 32 + threadIdx.x] = dw[i];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[i] += side[y * 256 + i * 32 + threadIdx.x];
    }
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (column<VEC>(c, i) < cols) out[column<VEC>(c, i)] = dw[i];
}

// The same with the rows' pieces 16-byte aligned and the whole row in one
// block (gridDim.y == 1), the next two rows on their way in.  DRAM bounds it:
// 8192 x 4096 bf16 rows with dh 45.4 us, 87% of the measured copy bandwidth,
// the reduction's launch included.
template <typename T, int VPT>
__global__ void __launch_bounds__(512)
    rmsnorm_grad_ring_kernel(const GradArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[128];
    const int threads = blockDim.x * blockDim.y;
    RowRing<T, 3, VPT> ring{ring_smem + threadIdx.y * blockDim.x + threadIdx.x};
    const int step = blockDim.x * 8, tid = threadIdx.x, cols = static_cast<int>(a.cols);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    auto fetch = [&](int64_t row, int slot) {
        if (row < a.rows) {
            ring.copy(slot, 0, static_cast<const T*>(a.dy) + row * a.lddy, step, tid, threads, cols);
            ring.copy(slot, 1, static_cast<const T*>(a.h) + row * a.ldh, step, tid, threads, cols);
            if (a.dh)
                ring.copy(slot, 2, static_cast<const T*>(a.dh) + row * a.lddh, step, tid, threads, cols);
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(row0 + i * stride, i);
    float dw[VPT][8], w[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        load8_any<true>(a.weight, a.weight_dtype, j * step + tid * 8, cols, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    }
    const float inv_n = 1.0f / static_cast<float>(cols);
    int slot = 0, turn = 0;
    for (int64_t row = row0; row < a.rows; row += stride, turn ^= 1) {
        const int refill = slot == 0 ? kRing - 1 : slot - 1;
        fetch(row + (kRing - 1) * stride, refill);
        ptx::cp_async_wait_groups<kRing - 1>();
        float s[2] = {0.0f, 0.0f};                 // sum h^2, sum dy w h
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float g[8], h[8];
            const bool in = j * step + tid * 8 < cols;
            ring.read(slot, 0, j, in, threads, g);
            ring.read(slot, 1, j, in, threads, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] += h[i] * h[i];
                s[1] += g[i] * w[j][i] * h[i];
            }
        }
        row_sum(s, slots, turn);
        const float rstd = rsqrtf(s[0] * inv_n + a.eps);
        const float back = s[1] * inv_n * rstd * rstd * rstd;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float g[8], h[8], o[8];
            const int c = j * step + tid * 8;
            ring.read(slot, 0, j, c < cols, threads, g);
            ring.read(slot, 1, j, c < cols, threads, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[i] *= rstd;
                o[i] = g[i] * w[j][i] - h[i] * back;
                dw[j][i] += g[i] * h[i];
            }
            if (a.dh) {
                float q[8];
                ring.read(slot, 2, j, c < cols, threads, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += q[i];
            }
            store8<T, true>(dx, c, cols, o);
        }
        if (++slot == kRing) slot = 0;
    }
    if (blockDim.y > 1) {                          // then blockDim.x == 32: one warp a row
        // The ring's memory takes the other warps' parts (it holds more).
        float* side = reinterpret_cast<float*>(ring_smem);
        __syncthreads();
        if (threadIdx.y > 0)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    side[(threadIdx.y - 1) * (VPT * 256) + (j * 8 + i) * 32 + tid] = dw[j][i];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dw[j][i] += side[y * (VPT * 256) + (j * 8 + i) * 32 + tid];
    }
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = j * step + tid * 8;
        if (c < cols)
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<float4*>(out + c + i) =
                    make_float4(dw[j][i], dw[j][i + 1], dw[j][i + 2], dw[j][i + 3]);
    }
}

struct QuantArgs {
    int64_t batch, rows, cols;
    const void* x;
    uint8_t* q;
    float* scales;
    int64_t ldx, stride_x, ldq, stride_q, scale_row, scale_col, scale_batch;
};

// One scale per row and 128 columns: 16 lanes a block of 128.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t nb = (a.cols + kBlock - 1) / kBlock;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
    const bool live = unit < a.batch * a.rows * nb;
    const int64_t row = live ? unit / nb : 0, t = live ? unit - row * nb : 0;
    const int64_t item = row / a.rows, r = row - item * a.rows;
    const int cols = static_cast<int>(a.cols);
    const int c = static_cast<int>(live ? t * kBlock + (threadIdx.x & 15) * 8 : nb * kBlock);   // past the end
    float v[8];
    load8<T, VEC>(static_cast<const T*>(a.x) + item * a.stride_x + r * a.ldx, c, cols, v);
    const float s = block_scale(block_amax(amax8(v))), inv = reciprocal(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    store8_e4m3<VEC>(a.q + item * a.stride_q + r * a.ldq, c, cols, v);
    if (live && (threadIdx.x & 15) == 0)
        a.scales[item * a.scale_batch + r * a.scale_row + t * a.scale_col] = s;
}

// One scale per 128 x 128: a block of 256 threads, 16 rows at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_square_kernel(const QuantArgs a) {
    __shared__ float best[8];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t nb = (a.cols + kBlock - 1) / kBlock, rb = (a.rows + kBlock - 1) / kBlock;
    const int64_t item = blockIdx.x / (nb * rb);
    const int64_t rest = blockIdx.x - item * nb * rb;
    const int64_t br = rest / nb, bc = rest - br * nb;
    const int cols = static_cast<int>(a.cols), past = static_cast<int>(nb * kBlock);
    const int c = static_cast<int>(bc * kBlock) + (threadIdx.x & 15) * 8;
    const T* x = static_cast<const T*>(a.x) + item * a.stride_x;
    float v[8][8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = br * kBlock + j * 16 + (threadIdx.x >> 4);
        load8<T, VEC>(x + r * a.ldx, r < a.rows ? c : past, cols, v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[j][i]));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, best[i]);
    const float s = block_scale(m), inv = reciprocal(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = br * kBlock + j * 16 + (threadIdx.x >> 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] *= inv;
        if (r < a.rows) store8_e4m3<VEC>(a.q + item * a.stride_q + r * a.ldq, c, cols, v[j]);
    }
    if (threadIdx.x == 0) a.scales[item * a.scale_batch + br * a.scale_row + bc * a.scale_col] = s;
}

constexpr int kRingVpt = 2;

template <typename T, bool FP8, bool RES>
int launch_norm_ring(const NormArgs& a, int threads, int sms, cudaStream_t st) {
    size_t smem = RowRing<T, RES ? 2 : 1, kRingVpt>::bytes(threads);
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e =
        opt_in_smem(rmsnorm_ring_kernel<T, kRingVpt, FP8, RES>, kRingBytesMost, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    // Blocks an SM: as many as it holds, but where residual rows stream through
    // DRAM only 512 threads, whose copies in flight saturate it with fewer
    // rows open at once: 16384 x 4096 bf16 rows (470 MB) 73.9 us against 86.9,
    // 8000 x 8192 71.9 against 82.8, while 11127 x 2728 (212 MB) takes 42.6
    // against 41.2.
    const bool stream = RES && a.rows * a.cols * static_cast<int64_t>(3 * sizeof(T) + 1) > (160ll << 20);
    const int per_sm = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(
        (stream ? 512 : 1536) / threads, 220 * 1024 / static_cast<int64_t>(smem + 1024))));
    if (stream) smem = std::max(smem, exact_smem(per_sm));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.rows, static_cast<int64_t>(sms) * per_sm)));
    return launch(rmsnorm_ring_kernel<T, kRingVpt, FP8, RES>, grid, dim3(threads), smem, st, a);
}

template <typename T, bool VEC, bool FP8>
int launch_norm(const NormArgs& a, cudaStream_t st) {
    const int64_t vectors = (a.cols + 7) / 8;
    // One vector a thread for as long as a block can hold the row: a row's loads
    // are then all in flight at once.
    int vpt = 1;
    while (vpt <= 4 && (vectors + vpt - 1) / vpt > kMaxThreads) vpt *= 2;
    if (vpt > 4) {
        return launch(rmsnorm_kernel<T, 0, VEC, FP8>, dim3(static_cast<unsigned>(a.rows)),
                      dim3(kMaxThreads, 1), 0, st, a);
    }
    const int threads = static_cast<int>(((vectors + vpt - 1) / vpt + 31) / 32 * 32);
    const int per_block = threads == 32 ? 8 : 1;
    const dim3 grid(static_cast<unsigned>((a.rows + per_block - 1) / per_block));
    const dim3 block(threads, per_block);
    switch (vpt) {
        case 1: return launch(rmsnorm_kernel<T, 1, VEC, FP8>, grid, block, 0, st, a);
        case 2: return launch(rmsnorm_kernel<T, 2, VEC, FP8>, grid, block, 0, st, a);
        default: return launch(rmsnorm_kernel<T, 4, VEC, FP8>, grid, block, 0, st, a);
    }
}

template <typename T>
int launch_norm_any(const NormArgs& a, bool vec, bool fp8, int sms, cudaStream_t st) {
    // The ring pays where rows are long (16384 x 256: 9.9 us against 5.7
    // without it, 16384 x 1024: 17.7 against 22.9) and 16-bit (fp32 pieces are
    // half a vector: 8000 x 4096 118 us against 76.7), and where there are more
    // rows than blocks.
    if constexpr (sizeof(T) == 2) {
        const int threads =
            static_cast<int>((a.cols + 32 * 8 * kRingVpt - 1) / (32 * 8 * kRingVpt) * 32);
        if (vec && threads > 32 && threads <= kRingThreads && a.rows > 2 * sms) {
            if (a.residual)
                return fp8 ? launch_norm_ring<T, true, true>(a, threads, sms, st)
                           : launch_norm_ring<T, false, true>(a, threads, sms, st);
            return fp8 ? launch_norm_ring<T, true, false>(a, threads, sms, st)
                       : launch_norm_ring<T, false, false>(a, threads, sms, st);
        }
    }
    if (vec) return fp8 ? launch_norm<T, true, true>(a, st) : launch_norm<T, true, false>(a, st);
    return fp8 ? launch_norm<T, false, true>(a, st) : launch_norm<T, false, false>(a, st);
}

constexpr int kGradVpt = 2;            // vectors a thread in the ring; one without it
constexpr int kGradRingThreads = 512;  // an SM

struct GradGeometry { int threads, per_block, blocks, per_sm, spans; };

// The blocks that sweep the rows, each of which writes one partial: as many as
// `threads_per_sm` allow, at most one per row (or eight rows of one warp).  The
// ring's copies in flight need no more than 512 threads an SM (8192 x 4096
// bf16 rows: 45 us, with 768 threads 51, with 1024 56); without the ring more
// threads hide the latency.
GradGeometry grad_geometry(int64_t rows, int64_t cols, int sms, bool ring) {
    GradGeometry g;
    const int vpt = ring ? kGradVpt : 1, threads_per_sm = ring ? kGradRingThreads : 1024;
    const int64_t vectors = (cols + 7) / 8;
    g.threads = static_cast<int>(std::min<int64_t>((vectors + 32 * vpt - 1) / (32 * vpt) * 32, 512));
    g.spans = static_cast<int>((vectors + vpt * g.threads - 1) / (vpt * g.threads));
    g.per_block = g.threads == 32 ? 8 : 1;
    const int64_t sweeps = (rows + g.per_block - 1) / g.per_block;
    g.per_sm = std::max(1, std::min(16, threads_per_sm / (g.threads * g.per_block)));
    g.blocks = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(sweeps, static_cast<int64_t>(sms) * g.per_sm)));
    return g;
}

// The 256-byte header and the partials of whichever form runs.
size_t grad_bytes(int64_t rows, int64_t cols, int sms) {
    const int blocks = std::max(grad_geometry(rows, cols, sms, true).blocks,
                                grad_geometry(rows, cols, sms, false).blocks);
    return kConvMinWorkspaceBytes + static_cast<size_t>(blocks) * static_cast<size_t>(cols) * 4;
}

template <typename T>
int launch_grad(const GradArgs& a, bool vec, int sms, int* parts, cudaStream_t st) {
    GradGeometry g = grad_geometry(a.rows, a.cols, sms, true);
    const size_t smem = RowRing<T, 3, kGradVpt>::bytes(g.threads * g.per_block);
    // fp32 pieces are half a vector, and fewer blocks fit beside their ring: only
    // while a block has few rows (fp32, 64 x 4096: 6.6 us against 9.5 without
    // the ring, 300 x 4096 9.7 against 11.3, 3187 x 1600 25.3 against 19.4).
    if (vec && g.spans == 1 && smem <= kRingBytesMost &&
        (sizeof(T) == 2 || a.rows <= 4 * sms)) {
        static std::atomic<uint64_t> opted{0};
        const cudaError_t e =
            opt_in_smem(rmsnorm_grad_ring_kernel<T, kGradVpt>, kRingBytesMost, &opted);
        if (e != cudaSuccess) return static_cast<int>(e);
        // fp32 rows take twice the shared memory: fewer blocks then.
        const int per_sm = std::max(
            1, std::min(g.per_sm, static_cast<int>(220 * 1024 / (smem + 1024))));
        *parts = std::min(g.blocks, sms * per_sm);
        return launch(rmsnorm_grad_ring_kernel<T, kGradVpt>, dim3(*parts),
                      dim3(g.threads, g.per_block), std::max(smem, exact_smem(per_sm)), st, a);
    }
    g = grad_geometry(a.rows, a.cols, sms, false);
    *parts = g.blocks;
    const dim3 grid(g.blocks, g.spans), block(g.threads, g.per_block);
    const size_t side = g.per_block > 1 ? (g.per_block - 1) * 256 * 4 : 0;
    if (g.spans > 1)
        return vec ? launch(rmsnorm_grad_kernel<T, true, true>, grid, block, side, st, a)
                   : launch(rmsnorm_grad_kernel<T, false, true>, grid, block, side, st, a);
    return vec ? launch(rmsnorm_grad_kernel<T, true, false>, grid, block, side, st, a)
               : launch(rmsnorm_grad_kernel<T, false, false>, grid, block, side, st, a);
}

template <typename T>
int launch_quantize(const QuantArgs& a, bool vec, bool square, cudaStream_t st) {
    const int64_t nb = (a.cols + kBlock - 1) / kBlock;
    const int64_t grid = square ? a.batch * ((a.rows + kBlock - 1) / kBlock) * nb
                                : (a.batch * a.rows * nb + 15) / 16;
    const dim3 g(static_cast<unsigned>(grid)), b(256);
    if (square)
        return vec ? launch(quantize_square_kernel<T, true>, g, b, 0, st, a)
                   : launch(quantize_square_kernel<T, false>, g, b, 0, st, a);
    return vec ? launch(quantize_rows_kernel<T, true>, g, b, 0, st, a)
               : launch(quantize_rows_kernel<T, false>, g, b, 0, st, a);
}

}  // namespace
}  // namespace tiles

using namespace tiles;

extern "C" {

int tiles_rmsnorm(const tiles_rmsnorm_desc* d, void* stream) {
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
    if ((s = check_matrix("x", d->x, d->ldx, d->cols, eb)) != TILES_OK) return s;
    if (d->residual && (s = check_matrix("residual", d->residual, d->ldr, d->cols, eb)) != TILES_OK)
        return s;
    if (d->h && (s = check_matrix("h", d->h, d->ldh, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("y", d->y, d->ldy, d->cols, fp8 ? 1 : eb)) != TILES_OK) return s;
    if (fp8 && (!d->scales || !element_aligned(d->scales, 4)))
        return fail(TILES_ERR_INVALID_ARG, "an e4m3 output needs aligned scales");
    NormArgs a{d->rows, d->cols, d->x, d->residual, d->weight, d->h, d->y, d->scales,
               d->ldx, d->ldr, d->ldh, d->ldy, d->scale_row, d->scale_block, d->eps,
               d->weight_dtype};
    const bool vec = d->cols % 8 == 0 && whole16(d->x, d->ldx, eb) &&
                     whole16(d->residual, d->ldr, eb) && whole16(d->h, d->ldh, eb) &&
                     whole16(d->weight, 0, 1) &&
                     (fp8 ? whole8(d->y, d->ldy) : whole16(d->y, d->ldy, eb));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    int e;
    if (d->dtype == TILES_BF16) e = launch_norm_any<__nv_bfloat16>(a, vec, fp8, sms, st);
    else if (d->dtype == TILES_F16) e = launch_norm_any<__half>(a, vec, fp8, sms, st);
    else e = launch_norm_any<float>(a, vec, fp8, sms, st);
    return launch_status(e, "norm");
}

size_t tiles_rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    if (check_sizes(rows, cols) != TILES_OK) return 0;
    int sms = 0;
    if (current_sm_count(&sms) != TILES_OK) return 0;
    return grad_bytes(rows, cols, sms);
}

int tiles_rmsnorm_grad(const tiles_rmsnorm_grad_desc* d, void* ws, size_t ws_bytes, void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_sizes(d->rows, d->cols);
    if (s != TILES_OK) return s;
    const int eb = dtype_bytes(d->dtype);
    if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "dy, h and dx must be f16, bf16 or f32");
    if (!d->dweight || !element_aligned(d->dweight, 4))
        return fail(TILES_ERR_INVALID_ARG, "dweight is null or not aligned to its element");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d->rows == 0) {
        const cudaError_t e = cudaMemsetAsync(d->dweight, 0, static_cast<size_t>(d->cols) * 4, st);
        return launch_status(e, "norm gradient");
    }
    if ((s = check_weight(d->weight, d->weight_dtype)) != TILES_OK) return s;
    if ((s = check_matrix("dy", d->dy, d->lddy, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("h", d->h, d->ldh, d->cols, eb)) != TILES_OK) return s;
    if (d->dh && (s = check_matrix("dh", d->dh, d->lddh, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("dx", d->dx, d->lddx, d->cols, eb)) != TILES_OK) return s;
    if (!ws) return fail(TILES_ERR_INVALID_ARG, "the norm gradient needs a workspace");
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(TILES_ERR_MISALIGNED, "the workspace must be 16-byte aligned");
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    const size_t need = grad_bytes(d->rows, d->cols, sms);
    if (ws_bytes < need)
        return fail(TILES_ERR_INVALID_ARG, "the norm gradient needs %zu workspace bytes", need);
    GradArgs a{d->rows, d->cols, d->dy, d->h, d->weight, d->dh, d->dx,
               reinterpret_cast<float*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes),
               d->lddy, d->ldh, d->lddh, d->lddx, d->eps, d->weight_dtype};
    const bool vec = d->cols % 8 == 0 && whole16(d->dy, d->lddy, eb) && whole16(d->h, d->ldh, eb) &&
                     whole16(d->dh, d->lddh, eb) && whole16(d->dx, d->lddx, eb) &&
                     whole16(d->weight, 0, 1);
    int e;
    int parts = 0;
    if (d->dtype == TILES_BF16) e = launch_grad<__nv_bfloat16>(a, vec, sms, &parts, st);
    else if (d->dtype == TILES_F16) e = launch_grad<__half>(a, vec, sms, &parts, st);
    else e = launch_grad<float>(a, vec, sms, &parts, st);
    if (e != cudaSuccess) return launch_status(e, "norm gradient");
    e = launch_reduce_partials(a.partials, d->cols, parts, d->dweight, nullptr, st);
    return launch_status(e, "norm gradient reduction");
}

int tiles_quantize_fp8(const tiles_quantize_desc* d, void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_sizes(d->rows, d->cols);
    if (s != TILES_OK) return s;
    if (d->batch < 0 || d->batch > kMaxRows) return fail(TILES_ERR_INVALID_ARG, "bad batch");
    const int eb = dtype_bytes(d->dtype);
    if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "x must be f16, bf16 or f32");
    if (d->block_rows != 1 && d->block_rows != 128)
        return fail(TILES_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (d->rows == 0 || d->batch == 0) return TILES_OK;
    if ((s = check_matrix("x", d->x, d->ldx, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("q", d->q, d->ldq, d->cols, 1)) != TILES_OK) return s;
    if (!d->scales || !element_aligned(d->scales, 4))
        return fail(TILES_ERR_INVALID_ARG, "scales is null or not aligned to its element");
    const int64_t nb = (d->cols + kBlock - 1) / kBlock;
    if (d->batch * ((d->rows + 15) / 16) > INT32_MAX / nb)
        return fail(TILES_ERR_TOO_LARGE, "too many blocks");
    QuantArgs a{d->batch, d->rows, d->cols, d->x, static_cast<uint8_t*>(d->q), d->scales, d->ldx,
                d->stride_x, d->ldq, d->stride_q, d->scale_row, d->scale_col, d->scale_batch};
    const bool vec = d->cols % 8 == 0 && whole16(d->x, d->ldx, eb) &&
                     d->stride_x * eb % 16 == 0 && whole8(d->q, d->ldq) && d->stride_q % 8 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool square = d->block_rows == 128;
    int e;
    if (d->dtype == TILES_BF16) e = launch_quantize<__nv_bfloat16>(a, vec, square, st);
    else if (d->dtype == TILES_F16) e = launch_quantize<__half>(a, vec, square, st);
    else e = launch_quantize<float>(a, vec, square, st);
    return launch_status(e, "quantise");
}

}  // extern "C"

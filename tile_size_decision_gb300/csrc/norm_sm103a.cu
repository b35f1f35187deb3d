// Root-mean-square norm with the residual's addition (16-bit, fp32 or scaled
// 8-bit output), its gradients, and the block quantiser of 8-bit matrices.
//
// All three read and write every element once and compute a few operations
// per byte: DRAM bounds them.  A row's elements stay in registers between
// the reduction and the output, so nothing is read twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>

#include "launch_util.h"
#include "sm103_ptx.cuh"
#include "tiles_internal.h"

namespace tiles {
namespace {

constexpr int kBlock = 128;             // columns that share one scale
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyScale = 0x1p-126f; // keeps the scale of a block of zeros usable
constexpr int kMaxThreads = 1024;

// fmaxf drops a NaN operand; a scale must keep it, or a row with a NaN would
// come out as finite numbers.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }

// Eight consecutive elements starting at column c (a multiple of 8).  With
// VEC they are whole 16-byte pieces; else each is loaded on its own, and
// those past the row's end read as zero.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t cols, float (&v)[8]) {
    if constexpr (VEC) {
        if (c < cols) {
            union { uint4 q[sizeof(T) / 2]; T e[8]; } u;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                u.q[i] = reinterpret_cast<const uint4*>(row + c)[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_float(u.e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float(row[c + i]) : 0.0f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int64_t c, int64_t cols, const float (&v)[8]) {
    if constexpr (VEC) {
        if (c < cols) {
            union { uint4 q[sizeof(T) / 2]; T e[8]; } u;
#pragma unroll
            for (int i = 0; i < 8; ++i) u.e[i] = from_float<T>(v[i]);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                reinterpret_cast<uint4*>(row + c)[i] = u.q[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = from_float<T>(v[i]);
    }
}

// The weight's type is its own; the branch is the same for every thread.
template <bool VEC>
__device__ __forceinline__ void load8_any(const void* p, int dtype, int64_t c, int64_t cols,
                                          float (&v)[8]) {
    if (dtype == TILES_BF16)
        load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(p), c, cols, v);
    else if (dtype == TILES_F16)
        load8<__half, VEC>(static_cast<const __half*>(p), c, cols, v);
    else
        load8<float, VEC>(static_cast<const float*>(p), c, cols, v);
}

// e4m3 of eight values over `scale`, as eight bytes.  The quotient's one
// rounding before the last is fp32's (a multiplication by the reciprocal).
template <bool VEC>
__device__ __forceinline__ void store8_e4m3(uint8_t* row, int64_t c, int64_t cols,
                                            const float (&v)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    if constexpr (VEC) {
        if (c < cols) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
    }
}

// Largest magnitude of the 128 values that 16 neighbouring lanes hold, eight
// each; columns past the row's end hold zeros.
__device__ __forceinline__ float block_amax(const float (&v)[8]) {
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

__device__ __forceinline__ float block_scale(float amax) {
    return max_nan(amax / kE4m3Max, kTinyScale);
}

// Sums over the threads of one row (blockDim.x threads, a multiple of 32);
// every thread gets them.  `slot` holds 2 x 32 floats per row of the block,
// used in turn, so that one barrier per call is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* slot, int turn) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], d);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    float* at = slot + turn * 32 * N;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int j = 0; j < N; ++j) at[j * 32 + (threadIdx.x >> 5)] = s[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float t = lane < warps ? at[j * 32 + lane] : 0.0f;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        s[j] = t;
    }
}

// ---- rows on their way in ----------------------------------------------------
//
// Rows whose pieces are 16-byte aligned come in through asynchronous copies,
// kRing rows deep.  A thread copies exactly the pieces it will read (its
// 8-element vectors of N matrices), so its own copy groups order them: no
// barrier, and no registers held by loads in flight.
constexpr int kRing = 3;

template <typename T, int N, int VPT>
struct RowRing {
    static constexpr int PIECES = static_cast<int>(sizeof(T)) / 2;   // 16-byte pieces of a vector
    static constexpr int STAGE = N * VPT * PIECES;                   // pieces per thread and row
    uint4* at;                                                       // + piece * threads

    static size_t bytes(int threads) {
        return static_cast<size_t>(kRing) * STAGE * threads * 16;
    }
    // Start the copies of matrix n's vectors for ring slot `slot`.
    __device__ __forceinline__ void copy(int slot, int n, const T* row, int step, int tid,
                                         int threads, int cols) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * step + tid * 8;
            if (c < cols)
#pragma unroll
                for (int p = 0; p < PIECES; ++p)
                    ptx::cp_async_16(at + ((slot * N + n) * VPT * PIECES + j * PIECES + p) * threads,
                                     reinterpret_cast<const uint4*>(row + c) + p);
        }
    }
    __device__ __forceinline__ void read(int slot, int n, int j, bool in, int threads,
                                         float (&v)[8]) const {
        union { uint4 q[PIECES]; T e[8]; } u;
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
            u.q[p] = in ? at[((slot * N + n) * VPT * PIECES + j * PIECES + p) * threads]
                        : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_float(u.e[i]);
    }
};

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
    auto load_h = [&](int64_t c, float (&v)[8]) {
        load8<T, VEC>(x, c, a.cols, v);
        if (r) {
            float q[8];
            load8<T, VEC>(r, c, a.cols, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
        }
    };
    auto emit = [&](int64_t c, const float (&v)[8], float rstd) {
        float w[8], y[8];
        load8_any<VEC>(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * rstd * w[i];
        if constexpr (FP8) {
            // Zeros past the row's end times rstd may be NaN; they must not
            // reach the short last block's scale.
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i >= a.cols) y[i] = 0.0f;
            const float s = block_scale(block_amax(y));
            store8_e4m3<VEC>(static_cast<uint8_t*>(a.y) + row * a.ldy, c, a.cols, y, 1.0f / s);
            if ((threadIdx.x & 15) == 0 && c < a.cols)
                a.scales[row * a.scale_row + c / kBlock * a.scale_block] = s;
        } else {
            store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy, c, a.cols, y);
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
            if (h) store8<T, VEC>(h, j * step + threadIdx.x * 8, a.cols, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[j][i] * v[j][i];
        }
        row_sum(sum, slots, 0);
        const float rstd = rsqrtf(sum[0] / static_cast<float>(a.cols) + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) emit(j * step + threadIdx.x * 8, v[j], rstd);
    } else {
        for (int64_t c0 = 0; c0 < a.cols; c0 += step) {
            float v[8];
            load_h(c0 + threadIdx.x * 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[i] * v[i];
        }
        row_sum(sum, slots, 0);
        const float rstd = rsqrtf(sum[0] / static_cast<float>(a.cols) + a.eps);
        for (int64_t c0 = 0; c0 < a.cols; c0 += step) {
            float v[8];
            load_h(c0 + threadIdx.x * 8, v);
            // h may be stored over x or the residual: after its own read.
            if (h) store8<T, VEC>(h, c0 + threadIdx.x * 8, a.cols, v);
            emit(c0 + threadIdx.x * 8, v, rstd);
        }
    }
}

// The same with the rows' pieces 16-byte aligned: the block takes rows
// blockIdx.x, + gridDim.x, ... (times blockDim.y), the next two of them on
// their way in while one is worked on.
template <typename T, int VPT, bool FP8>
__global__ void __launch_bounds__(kMaxThreads)
    rmsnorm_ring_kernel(const NormArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[64];
    const int threads = blockDim.x * blockDim.y;
    RowRing<T, 2, VPT> ring{ring_smem + threadIdx.y * blockDim.x + threadIdx.x};
    const int step = blockDim.x * 8, tid = threadIdx.x, cols = static_cast<int>(a.cols);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    auto fetch = [&](int64_t row, int slot) {
        if (row < a.rows) {
            ring.copy(slot, 0, static_cast<const T*>(a.x) + row * a.ldx, step, tid, threads, cols);
            if (a.residual)
                ring.copy(slot, 1, static_cast<const T*>(a.residual) + row * a.ldr, step, tid, threads,
                          cols);
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(row0 + i * stride, i);
    int slot = 0, turn = 0;
    for (int64_t row = row0; row < a.rows; row += stride, turn ^= 1) {
        const int refill = slot == 0 ? kRing - 1 : slot - 1;
        fetch(row + (kRing - 1) * stride, refill);
        ptx::cp_async_wait_groups<kRing - 1>();
        float v[VPT][8], sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * step + tid * 8;
            ring.read(slot, 0, j, c < cols, threads, v[j]);
            if (a.residual) {
                float q[8];
                ring.read(slot, 1, j, c < cols, threads, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] += q[i];
            }
            if (a.h) store8<T, true>(static_cast<T*>(a.h) + row * a.ldh, c, cols, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] += v[j][i] * v[j][i];
        }
        row_sum(sum, slots, turn);
        const float rstd = rsqrtf(sum[0] / static_cast<float>(cols) + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * step + tid * 8;
            float w[8], y[8];
            load8_any<true>(a.weight, a.weight_dtype, c, cols, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = c < cols ? v[j][i] * rstd * w[i] : 0.0f;
            if constexpr (FP8) {
                const float s = block_scale(block_amax(y));
                store8_e4m3<true>(static_cast<uint8_t*>(a.y) + row * a.ldy, c, cols, y, 1.0f / s);
                if ((tid & 15) == 0 && c < cols)
                    a.scales[row * a.scale_row + c / kBlock * a.scale_block] = s;
            } else {
                store8<T, true>(static_cast<T*>(a.y) + row * a.ldy, c, cols, y);
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
// columns when a row is longer than one block's registers hold (VPT vectors
// a thread): each span then reads the whole row for the two sums and writes
// its own columns.
template <typename T, int VPT, bool VEC>
__global__ void __launch_bounds__(512)
    rmsnorm_grad_kernel(const GradArgs a) {
    __shared__ float slots[128];
    __shared__ float side[7][VPT * 256];           // blockDim.y > 1: the other warps' parts
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int step = blockDim.x * 8;
    const int64_t first = static_cast<int64_t>(blockIdx.y) * VPT * step;
    float dw[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * blockDim.y, turn ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* h = static_cast<const T*>(a.h) + row * a.ldh;
        float g[VPT][8], v[VPT][8];
        float s[2] = {0.0f, 0.0f};                 // sum h^2, sum dy w h
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int64_t c = first + j * step + threadIdx.x * 8;
            load8<T, VEC>(dy, c, a.cols, g[j]);
            load8<T, VEC>(h, c, a.cols, v[j]);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float w[8];
            load8_any<VEC>(a.weight, a.weight_dtype, first + j * step + threadIdx.x * 8, a.cols, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] += v[j][i] * v[j][i];
                s[1] += g[j][i] * w[i] * v[j][i];
            }
        }
        if (gridDim.y > 1) {
            for (int64_t c0 = 0; c0 < a.cols; c0 += step) {
                if (c0 >= first && c0 < first + VPT * step) continue;
                const int64_t c = c0 + threadIdx.x * 8;
                float p[8], q[8], w[8];
                load8<T, VEC>(dy, c, a.cols, p);
                load8<T, VEC>(h, c, a.cols, q);
                load8_any<VEC>(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[0] += q[i] * q[i];
                    s[1] += p[i] * w[i] * q[i];
                }
            }
        }
        row_sum(s, slots, turn);
        const float inv_n = 1.0f / static_cast<float>(a.cols);
        const float rstd = rsqrtf(s[0] * inv_n + a.eps);
        const float back = s[1] * inv_n * rstd * rstd * rstd;
        const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int64_t c = first + j * step + threadIdx.x * 8;
            float w[8], o[8];
            load8_any<VEC>(a.weight, a.weight_dtype, c, a.cols, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = g[j][i] * w[i] * rstd - v[j][i] * back;
                dw[j][i] += g[j][i] * v[j][i] * rstd;
            }
            if (dh) {
                float q[8];
                load8<T, VEC>(dh, c, a.cols, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += q[i];
            }
            store8<T, VEC>(dx, c, a.cols, o);
        }
    }
    if (blockDim.y > 1) {                          // then blockDim.x == 32: one warp a row
        if (threadIdx.y > 0)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    side[threadIdx.y - 1][(j * 8 + i) * 32 + threadIdx.x] = dw[j][i];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[j][i] += side[y][(j * 8 + i) * 32 + threadIdx.x];
    }
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int64_t c = first + j * step + threadIdx.x * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < a.cols) out[c + i] = dw[j][i];
    }
}

// The same with the rows' pieces 16-byte aligned and the whole row in one
// block (gridDim.y == 1), the next two rows on their way in.
template <typename T, int VPT>
__global__ void __launch_bounds__(512)
    rmsnorm_grad_ring_kernel(const GradArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[128];
    __shared__ float side[7][VPT * 256];           // blockDim.y > 1: the other warps' parts
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
        if (threadIdx.y > 0)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) side[threadIdx.y - 1][(j * 8 + i) * 32 + tid] = dw[j][i];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[j][i] += side[y][(j * 8 + i) * 32 + tid];
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

// dweight[c] = the sum of the partials of column c: 32 columns a block, 32
// threads a column, each over every 32nd partial, added in a fixed order.
__global__ void __launch_bounds__(1024) reduce_partials_kernel(const float* partials, int64_t cols,
                                                               int parts, float* out) {
    __shared__ float s[32][33];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float t = 0.0f;
    if (c < cols)
        for (int p = threadIdx.y; p < parts; p += 32) t += partials[p * cols + c];
    s[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
#pragma unroll
        for (int j = 1; j < 32; ++j) t += s[j][threadIdx.x];
        out[c] = t;
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
    const int64_t c = live ? t * kBlock + (threadIdx.x & 15) * 8 : a.cols;
    float v[8];
    load8<T, VEC>(static_cast<const T*>(a.x) + item * a.stride_x + r * a.ldx, c, a.cols, v);
    const float s = block_scale(block_amax(v));
    store8_e4m3<VEC>(a.q + item * a.stride_q + r * a.ldq, c, a.cols, v, 1.0f / s);
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
    const int64_t c = bc * kBlock + (threadIdx.x & 15) * 8;
    const T* x = static_cast<const T*>(a.x) + item * a.stride_x;
    float v[8][8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = br * kBlock + j * 16 + (threadIdx.x >> 4);
        load8<T, VEC>(x + r * a.ldx, r < a.rows ? c : a.cols, a.cols, v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[j][i]));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, best[i]);
    const float s = block_scale(m), inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = br * kBlock + j * 16 + (threadIdx.x >> 4);
        if (r < a.rows)
            store8_e4m3<VEC>(a.q + item * a.stride_q + r * a.ldq, c, a.cols, v[j], inv);
    }
    if (threadIdx.x == 0) a.scales[item * a.scale_batch + br * a.scale_row + bc * a.scale_col] = s;
}

bool whole16(const void* p, int64_t pitch_elems, int elem_bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 &&
                            pitch_elems * elem_bytes % 16 == 0);
}

bool whole8(const void* p, int64_t pitch_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & 7u) == 0 && pitch_bytes % 8 == 0;
}

bool element_aligned(const void* p, int elem_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem_bytes - 1)) == 0;
}

#ifndef NTH
#define NTH 1536
#endif
constexpr int kRingBytesMost = 96 * 1024;            // two blocks an SM

template <typename T, int VPT, bool FP8>
int launch_norm_ring(const NormArgs& a, int sms, cudaStream_t st) {
    const int64_t vectors = (a.cols + 7) / 8;
    const int threads = static_cast<int>((vectors + 32 * VPT - 1) / (32 * VPT) * 32);
    const int per_block = threads == 32 ? 8 : 1;
    const size_t smem = RowRing<T, 2, VPT>::bytes(threads * per_block);
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(rmsnorm_ring_kernel<T, VPT, FP8>, kRingBytesMost, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    // As many blocks as an SM holds (threads and shared memory).
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(
        NTH / (threads * per_block), 220 * 1024 / static_cast<int64_t>(smem + 1024)));
    const int64_t need = (a.rows + per_block - 1) / per_block;
    const dim3 grid(static_cast<unsigned>(std::min(need, sms * per_sm)));
    return launch(rmsnorm_ring_kernel<T, VPT, FP8>, grid, dim3(threads, per_block), smem, st, a);
}

template <typename T, bool VEC, bool FP8>
int launch_norm(const NormArgs& a, cudaStream_t st) {
    const int64_t vectors = (a.cols + 7) / 8;
    // One 8-element vector a thread for as long as a block can hold the row: a row's
    // loads are then all in flight at once.
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
    const int64_t vectors = (a.cols + 7) / 8;
    int v = 2; if (getenv("VPT")) v = atoi(getenv("VPT"));
    if (vec && vectors <= 2048 && v && RowRing<T, 2, 2>::bytes((vectors + 63) / 64 * 32) <= kRingBytesMost) {
        if (v == 2) return fp8 ? launch_norm_ring<T, 2, true>(a, sms, st) : launch_norm_ring<T, 2, false>(a, sms, st);
        if (v == 4) return fp8 ? launch_norm_ring<T, 4, true>(a, sms, st) : launch_norm_ring<T, 4, false>(a, sms, st);
        if (v == 1) return fp8 ? launch_norm_ring<T, 1, true>(a, sms, st) : launch_norm_ring<T, 1, false>(a, sms, st);
    }
    if (vec) return fp8 ? launch_norm<T, true, true>(a, st) : launch_norm<T, true, false>(a, st);
    return fp8 ? launch_norm<T, false, true>(a, st) : launch_norm<T, false, false>(a, st);
}

#ifndef GV
#define GV 2
#define GC 512
#endif
constexpr int kGradVpt = GV;

struct GradGeometry { int threads, per_block, blocks, spans; };

// The blocks that sweep the rows: as many as are resident at once, so that
// each writes one partial; at most one per row.
GradGeometry grad_geometry(int64_t rows, int64_t cols, int sms) {
    GradGeometry g;
    const int64_t vectors = (cols + 7) / 8;
    const int64_t per_block = (vectors + kGradVpt - 1) / kGradVpt;
    g.threads = static_cast<int>(std::min<int64_t>((per_block + 31) / 32 * 32, 512));
    g.spans = static_cast<int>((vectors + kGradVpt * g.threads - 1) / (kGradVpt * g.threads));
    g.per_block = g.threads == 32 ? 8 : 1;
    const int64_t resident =
        static_cast<int64_t>(sms) * std::max(1, std::min(8, GC / (g.threads * g.per_block)));
    g.blocks = static_cast<int>(
        std::max<int64_t>(1, std::min((rows + g.per_block - 1) / g.per_block, resident)));
    return g;
}

template <typename T>
int launch_grad(const GradArgs& a, bool vec, const GradGeometry& g, cudaStream_t st) {
    const dim3 grid(g.blocks, g.spans), block(g.threads, g.per_block);
    const size_t smem = RowRing<T, 3, kGradVpt>::bytes(g.threads * g.per_block);
    if (vec && g.spans == 1 && smem <= kRingBytesMost && !getenv("NORING")) {
        static std::atomic<uint64_t> opted{0};
        const cudaError_t e =
            opt_in_smem(rmsnorm_grad_ring_kernel<T, kGradVpt>, kRingBytesMost, &opted);
        if (e != cudaSuccess) return static_cast<int>(e);
        return launch(rmsnorm_grad_ring_kernel<T, kGradVpt>, grid, block, smem, st, a);
    }
    return vec ? launch(rmsnorm_grad_kernel<T, kGradVpt, true>, grid, block, 0, st, a)
               : launch(rmsnorm_grad_kernel<T, kGradVpt, false>, grid, block, 0, st, a);
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

int check_matrix(const char* what, const void* p, int64_t ld, int64_t cols, int elem_bytes) {
    if (!p) return fail(TILES_ERR_INVALID_ARG, "%s is null", what);
    if (ld < cols) return fail(TILES_ERR_INVALID_ARG, "%s: row pitch smaller than the row length", what);
    if (!element_aligned(p, elem_bytes))
        return fail(TILES_ERR_MISALIGNED, "%s is not aligned to its element", what);
    return TILES_OK;
}

constexpr int64_t kMaxRows = INT32_MAX / 2;

int check_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1)
        return fail(TILES_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (rows=%lld cols=%lld)",
                    (long long)rows, (long long)cols);
    if (rows > kMaxRows || cols > kMaxRows) return fail(TILES_ERR_TOO_LARGE, "a size exceeds 2^30");
    return TILES_OK;
}

int check_weight(const void* w, int dtype) {
    const int wb = dtype_bytes(dtype);
    if (!wb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the weight must be f16, bf16 or f32");
    if (!w) return fail(TILES_ERR_INVALID_ARG, "weight is null");
    if (!element_aligned(w, wb))
        return fail(TILES_ERR_MISALIGNED, "weight is not aligned to its element");
    return TILES_OK;
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
    const GradGeometry g = grad_geometry(rows, cols, sms);
    return kConvMinWorkspaceBytes + static_cast<size_t>(g.blocks) * cols * 4;
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
    const GradGeometry g = grad_geometry(d->rows, d->cols, sms);
    const size_t need = kConvMinWorkspaceBytes + static_cast<size_t>(g.blocks) * d->cols * 4;
    if (ws_bytes < need)
        return fail(TILES_ERR_INVALID_ARG, "the norm gradient needs %zu workspace bytes", need);
    GradArgs a{d->rows, d->cols, d->dy, d->h, d->weight, d->dh, d->dx,
               reinterpret_cast<float*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes),
               d->lddy, d->ldh, d->lddh, d->lddx, d->eps, d->weight_dtype};
    const bool vec = d->cols % 8 == 0 && whole16(d->dy, d->lddy, eb) && whole16(d->h, d->ldh, eb) &&
                     whole16(d->dh, d->lddh, eb) && whole16(d->dx, d->lddx, eb) &&
                     whole16(d->weight, 0, 1);
    int e;
    if (d->dtype == TILES_BF16) e = launch_grad<__nv_bfloat16>(a, vec, g, st);
    else if (d->dtype == TILES_F16) e = launch_grad<__half>(a, vec, g, st);
    else e = launch_grad<float>(a, vec, g, st);
    if (e != cudaSuccess) return launch_status(e, "norm gradient");
    e = launch(reduce_partials_kernel, dim3(static_cast<unsigned>((d->cols + 31) / 32)),
               dim3(32, 32), 0, st, static_cast<const float*>(a.partials), d->cols, g.blocks,
               d->dweight);
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

// What the row operators (norms, their gradients, the quantiser) share: rows
// of 16-bit or fp32 elements in registers, scaled 8-bit stores, sums over a
// row's threads, rows on their way in through shared memory, the addition of
// partial gradients, and the checks of the calls' arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch_util.h"
#include "op_ptx.cuh"
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

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The larger magnitude of three, NaN if one is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// Two fp32 values as a packed pair of T, and back (T of 16 bits).
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Eight elements as they lie in memory (16-byte pieces) as fp32.
template <typename T>
__device__ __forceinline__ void widen8(const uint4 (&q)[sizeof(T) / 2], float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            v[4 * p] = __uint_as_float(q[p].x);
            v[4 * p + 1] = __uint_as_float(q[p].y);
            v[4 * p + 2] = __uint_as_float(q[p].z);
            v[4 * p + 3] = __uint_as_float(q[p].w);
        }
    } else {
        const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = unpack2<T>(w[i]);
            v[2 * i] = t.x;
            v[2 * i + 1] = t.y;
        }
    }
}

// A thread's "vector" c (a multiple of 8) is eight columns.  With VEC they
// are consecutive, whole 16-byte pieces.  Without (rows that start anywhere)
// each element moves on its own, and the 16 threads of a block of 128 columns
// take every 16th column of it, so that neighbours touch neighbours; columns
// past the row's end read as zero.
template <bool VEC>
__device__ __forceinline__ int column(int c, int i) {
    return VEC ? c + i : (c & ~127) + ((c >> 3) & 15) + 16 * i;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int cols, float (&v)[8]) {
    if constexpr (VEC) {
        uint4 q[sizeof(T) / 2];
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            q[i] = c < cols ? reinterpret_cast<const uint4*>(row + c)[i] : make_uint4(0, 0, 0, 0);
        widen8<T>(q, v);
    } else {
        const T* at = row + column<false>(c, 0);
        if ((c | 127) < cols) {                       // the whole block is inside the row
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_float(at[16 * i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = column<false>(c, i) < cols ? to_float(at[16 * i]) : 0.0f;
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int c, int cols, const float (&v)[8]) {
    if constexpr (VEC) {
        if (c >= cols) return;
        uint4* to = reinterpret_cast<uint4*>(row + c);
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *to = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                             pack2<T>(v[6], v[7]));
        }
    } else {
        T* at = row + column<false>(c, 0);
        if ((c | 127) < cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) at[16 * i] = from_float<T>(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (column<false>(c, i) < cols) at[16 * i] = from_float<T>(v[i]);
        }
    }
}

// The weight's type is its own; the branch is the same for every thread.
template <bool VEC>
__device__ __forceinline__ void load8_any(const void* p, int dtype, int c, int cols,
                                          float (&v)[8]) {
    if (dtype == TILES_BF16)
        load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(p), c, cols, v);
    else if (dtype == TILES_F16)
        load8<__half, VEC>(static_cast<const __half*>(p), c, cols, v);
    else
        load8<float, VEC>(static_cast<const float*>(p), c, cols, v);
}

// Eight values, already over their scale, as e4m3 bytes.
template <bool VEC>
__device__ __forceinline__ void store8_e4m3(uint8_t* row, int c, int cols, const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    if constexpr (VEC) {
        if (c < cols) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (column<false>(c, i) < cols)
                row[column<false>(c, i)] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
    }
}

// Largest magnitude of a thread's eight values, and of the 128 that 16
// neighbouring lanes hold; columns past the row's end hold zeros.
__device__ __forceinline__ float amax8(const float (&v)[8]) {
    const float m = max3_abs_nan(max3_abs_nan(v[0], v[1], v[2]), v[3], v[4]);
    return max3_abs_nan(max3_abs_nan(m, v[5], v[6]), v[7], 0.0f);
}

__device__ __forceinline__ float block_amax(float m) {
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

__device__ __forceinline__ float block_scale(float amax) {
    return max_nan(amax * (1.0f / kE4m3Max), kTinyScale);
}

// 1 / scale: scales are normal numbers, so the hardware's approximation (one
// unit in the last place) is enough before a rounding to four bits.
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
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

// The bytes of what is read.
struct Extent {
    const char* from;
    const char* to;                           // past the last
};

// The bytes of a matrix's rows.
template <typename T>
__device__ __forceinline__ Extent extent_of(const void* p, int64_t rows, int64_t ld, int64_t cols) {
    const char* at = static_cast<const char*>(p);
    return {at, at + ((rows - 1) * ld + cols) * static_cast<int64_t>(sizeof(T))};
}

// 16 bytes that start on any element, inside the extent: the two aligned pieces that
// hold them as they lie in memory, so that many can be asked for before the first one is
// looked at, and then what starts `shift` bytes into them.
struct Window {
    uint4 lo, hi;
    int shift;

    __device__ __forceinline__ void load(const char* p, const Extent& e, int elem_bytes) {
        shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
        const char* base = p - shift;
        if (base >= e.from && base + 32 <= e.to) {
            lo = *reinterpret_cast<const uint4*>(base);
            hi = *reinterpret_cast<const uint4*>(base + 16);
        } else {
            // At the ends the aligned pieces may reach out of the extent.
            lo = hi = by_element(p, elem_bytes);
            shift = 0;
        }
    }
    static __device__ __forceinline__ uint4 by_element(const char* p, int elem_bytes) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (elem_bytes == 4) {
                w[i] = reinterpret_cast<const uint32_t*>(p)[i];
            } else if (elem_bytes == 2) {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + 2 * i;
                w[i] = q[0] | static_cast<uint32_t>(q[1]) << 16;
            } else {
                const uint8_t* q = reinterpret_cast<const uint8_t*>(p) + 4 * i;
                w[i] = q[0] | static_cast<uint32_t>(q[1]) << 8 | static_cast<uint32_t>(q[2]) << 16 |
                       static_cast<uint32_t>(q[3]) << 24;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 get() const {
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
        const int bits = (shift & 3) * 8;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
};

// The same at once.
__device__ __forceinline__ uint4 unaligned16(const char* p, const Extent& e, int elem_bytes) {
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) return *reinterpret_cast<const uint4*>(p);
    Window w;
    w.load(p, e, elem_bytes);
    return w.get();
}

// Lane l's share of the warp's sums of s[0 .. N): that of s[l % N].  Each exchange
// halves what a lane is responsible for; of the N values the last N - USED
// are zeros.
template <int N, int USED>
__device__ __forceinline__ float fold(float (&s)[N]) {
    const int lane = threadIdx.x & 31;
    int live = USED;
#pragma unroll
    for (int bit = 1; bit < N; bit <<= 1) {
#pragma unroll
        for (int i = 0; i < N / 2 / bit; ++i)
            if (2 * i < live) {
                const float lo = s[2 * i], hi = 2 * i + 1 < live ? s[2 * i + 1] : 0.0f;
                s[i] = (lane & bit ? hi : lo) + __shfl_xor_sync(0xffffffffu, lane & bit ? lo : hi, bit);
            }
        live = (live + 1) / 2;
    }
    float x = s[0];
#pragma unroll
    for (int d = N; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// ---- rows on their way in ----------------------------------------------------
//
// Rows whose pieces are 16-byte aligned come in through asynchronous copies,
// kRing rows deep.  A thread copies exactly the pieces it will read (its
// 8-element vectors of N matrices), so its own copy groups order them: no
// barrier, and no registers held by loads in flight.
constexpr int kRing = 3;
constexpr int kRingThreads = 512;

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
        uint4 q[PIECES];
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
            q[p] = in ? at[((slot * N + n) * VPT * PIECES + j * PIECES + p) * threads]
                      : make_uint4(0, 0, 0, 0);
        widen8<T>(q, v);
    }
};

// out[c] = the sum of the partials of column c: COLUMNS columns a block, R threads
// a column, each over every R-th partial, then a tree: a fixed order, which is the
// same for every R that is no less than the partials are.
// Partials of two gradients lie side by side ([parts][2][cols], gridDim.y 2).
template <int COLUMNS, int R>
__global__ void __launch_bounds__(COLUMNS * R) reduce_partials_kernel(const float* partials, int64_t cols,
                                                                      int parts, float* out, float* out2) {
    __shared__ float s[R][COLUMNS + 1];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * COLUMNS + threadIdx.x;
    const int64_t pitch = cols * gridDim.y, at = c + cols * blockIdx.y;
    float t = 0.0f;
    if (c < cols)
#pragma unroll 4
        for (int p = threadIdx.y; p < parts; p += R) t += partials[p * pitch + at];
    s[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
#pragma unroll
    for (int d = R / 2; d >= 1; d >>= 1) {
        if (static_cast<int>(threadIdx.y) < d)
            s[threadIdx.y][threadIdx.x] += s[threadIdx.y + d][threadIdx.x];
        __syncthreads();
    }
    if (threadIdx.y == 0 && c < cols) (blockIdx.y ? out2 : out)[c] = s[0][threadIdx.x];
}

// ---- the host's side -----------------------------------------------------------

template <int COLUMNS, int R>
int launch_reduce_partials_of(const float* partials, int64_t cols, int parts, float* out, float* out2,
                              cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((cols + COLUMNS - 1) / COLUMNS), out2 ? 2 : 1);
    return launch(reduce_partials_kernel<COLUMNS, R>, grid, dim3(COLUMNS, R), 0, st, partials, cols, parts, out,
                  out2);
}

// 64 threads a column (with 32 columns a block, 1024 columns kept only 32 SMs busy:
// 28.2 us for the root-mean-square norm's gradient of 16384 x 1024 rows against 26.8; with
// 8, 41.5 us against 39.0 for 3000 x 8192); few partials want no more threads than
// they are (1 row of 8192 columns 7.0 us against 11.1, 16 of 3200 5.8 against 7.5).  Of
// two gradients, whose blocks are twice as many, 32 threads a column until the partials
// are many (layer norm's gradient, 3000 x 8192 46.4 us against 51.8, 8192 x 4096 53.8
// against 56.5; 1718 x 637, where they are 1520, 17.1 against 15.1).
inline int launch_reduce_partials(const float* partials, int64_t cols, int parts, float* out,
                                  float* out2, cudaStream_t st) {
    if (parts <= 8) return launch_reduce_partials_of<32, 8>(partials, cols, parts, out, out2, st);
    if (parts <= 32 || (out2 && parts <= 512)) return launch_reduce_partials_of<16, 32>(partials, cols, parts, out, out2, st);
    return launch_reduce_partials_of<16, 64>(partials, cols, parts, out, out2, st);
}

inline bool whole16(const void* p, int64_t pitch_elems, int elem_bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 &&
                            pitch_elems * elem_bytes % 16 == 0);
}

inline bool whole8(const void* p, int64_t pitch_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & 7u) == 0 && pitch_bytes % 8 == 0;
}

inline bool element_aligned(const void* p, int elem_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem_bytes - 1)) == 0;
}

constexpr int kRingBytesMost = 200 * 1024;

// Dynamic shared memory that lets exactly `per_sm` blocks on an SM (228 KB, of
// which each block costs 1 KB more than it asks for): a persistent grid of that
// many blocks an SM is then spread evenly, also while the kernel before it
// still holds some SMs.
inline size_t exact_smem(int per_sm) {
    return std::min<size_t>(static_cast<size_t>(228 * 1024 / (per_sm + 1)), kRingBytesMost);
}

inline int check_matrix(const char* what, const void* p, int64_t ld, int64_t cols, int elem_bytes) {
    if (!p) return fail(TILES_ERR_INVALID_ARG, "%s is null", what);
    if (ld < cols) return fail(TILES_ERR_INVALID_ARG, "%s: row pitch smaller than the row length", what);
    if (!element_aligned(p, elem_bytes))
        return fail(TILES_ERR_MISALIGNED, "%s is not aligned to its element", what);
    return TILES_OK;
}

constexpr int64_t kMaxRows = INT32_MAX / 2;

inline int check_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1)
        return fail(TILES_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (rows=%lld cols=%lld)",
                    (long long)rows, (long long)cols);
    if (rows > kMaxRows || cols > kMaxRows) return fail(TILES_ERR_TOO_LARGE, "a size exceeds 2^30");
    return TILES_OK;
}

inline int check_weight(const void* w, int dtype) {
    const int wb = dtype_bytes(dtype);
    if (!wb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the weight must be f16, bf16 or f32");
    if (!w) return fail(TILES_ERR_INVALID_ARG, "weight is null");
    if (!element_aligned(w, wb))
        return fail(TILES_ERR_MISALIGNED, "weight is not aligned to its element");
    return TILES_OK;
}

}  // namespace
}  // namespace tiles

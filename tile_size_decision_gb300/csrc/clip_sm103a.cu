// The common norm of many gradients, and their scaling by it.
//
// The norm reads every element once, the scaling reads and writes every
// element once: DRAM bounds both, and launches where the gradients are small.
#include <algorithm>
#include <cfloat>
#include <exception>
#include <vector>

#include "row_ops.cuh"

namespace tiles {
namespace {

// Tensors a launch takes: their descriptions travel with it as arguments (4 KB),
// so that nothing on the host has to outlive the call and a captured launch
// carries them.
constexpr int kTensors = 120;
constexpr int kClipThreads = 256;
constexpr int kClipBlocksPerSm = 8;

struct Tensor {
    const void* from;
    void* to;
    int64_t count;
    int32_t dtype;
    uint32_t chunks_before;                    // of the launch's tensors before this one
};

struct TensorBatch {
    int32_t tensors;
    uint32_t chunks;
    int32_t parts;                             // partial sums in all, of all launches
    float max_norm, eps;
    int32_t pad0;
    double* partials;                          // this launch's first, or (scaling) the very first
    float* norm;
    Tensor at[kTensors];
};
static_assert(sizeof(TensorBatch) <= 4096, "arguments of one launch");

// Bytes of one chunk, the share of a tensor that a block takes at a time: U
// 16-byte pieces a thread.
template <int U> constexpr int kChunkBytes = U * kClipThreads * 16;

// Squares and sums in fp32 within a thread's pieces of a chunk, in fp64 from
// there on.  Where that leaves fp32's range (a square over 2^127, or squares
// that together are under 2^-90 and are not of zeros) the thread takes its
// elements once more in fp64.
constexpr float kSmallSquares = 0x1p-90f;

template <typename T> __device__ __forceinline__ constexpr uint32_t magnitude_bits() {
    return sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
}

template <typename T>
__device__ __forceinline__ void widen_piece(uint4 q, float (&v)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(q.x);
        v[1] = __uint_as_float(q.y);
        v[2] = __uint_as_float(q.z);
        v[3] = __uint_as_float(q.w);
    } else {
        const uint4 p[1] = {q};
        widen8<T>(p, v);
    }
}

template <typename T>
__device__ __noinline__ double squares_in_double(const uint4* q, int pieces) {
    double s = 0.0;
    for (int u = 0; u < pieces; ++u) {
        float v[16 / sizeof(T)];
        widen_piece<T>(q[u], v);
        for (float e : v) s += static_cast<double>(e) * static_cast<double>(e);
    }
    return s;
}

// The squares of a thread's share of the chunk that starts at element `first`.
template <typename T, int U>
__device__ __forceinline__ double chunk_squares(const Tensor& t, int64_t first) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const T* from = static_cast<const T*>(t.from) + first;
    const int64_t left = t.count - first;
    uint4 q[U];
    if (left >= kChunkBytes<U> / static_cast<int>(sizeof(T)) &&
        (reinterpret_cast<uintptr_t>(t.from) & 15u) == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            q[u] = reinterpret_cast<const uint4*>(from)[u * kClipThreads + threadIdx.x];
    } else {
        // A tensor's last chunk, and tensors that start anywhere: element by
        // element, neighbours on neighbours; zeros past the end.
#pragma unroll
        for (int u = 0; u < U; ++u) {
            T e[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t at = static_cast<int64_t>(u * N + i) * kClipThreads + threadIdx.x;
                e[i] = at < left ? from[at] : from_float<T>(0.0f);
            }
            memcpy(&q[u], e, 16);
        }
    }
    float s = 0.0f;
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        any |= q[u].x | q[u].y | q[u].z | q[u].w;
        float v[N];
        widen_piece<T>(q[u], v);
#pragma unroll
        for (int i = 0; i < N; ++i) s += v[i] * v[i];
    }
    if (!(s >= kSmallSquares && s <= FLT_MAX) && (any & magnitude_bits<T>()))
        return squares_in_double<T>(q, U);
    return static_cast<double>(s);
}

// The sum over a block; every thread gets it.
__device__ __forceinline__ double block_sum(double s) {
    __shared__ double warp_sums[kClipThreads / 32];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int i = 0; i < kClipThreads / 32; ++i) s += warp_sums[i];
    return s;
}

// One partial sum a block, over the chunks blockIdx.x, + gridDim.x, ...
template <int U>
__global__ void __launch_bounds__(kClipThreads) squares_kernel(const __grid_constant__ TensorBatch a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    double s = 0.0;
    int n = 0;
    for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        while (n + 1 < a.tensors && c >= a.at[n + 1].chunks_before) ++n;
        const Tensor& t = a.at[n];
        const int64_t bytes = static_cast<int64_t>(c - t.chunks_before) * kChunkBytes<U>;
        if (t.dtype == TILES_BF16) s += chunk_squares<__nv_bfloat16, U>(t, bytes / 2);
        else if (t.dtype == TILES_F16) s += chunk_squares<__half, U>(t, bytes / 2);
        else s += chunk_squares<float, U>(t, bytes / 4);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
}

// The norm from all partial sums, in a fixed order (every thread of a block
// gets it).
__device__ __forceinline__ float norm_of(const double* partials, int parts) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) s += partials[i];
    return static_cast<float>(sqrt(block_sum(s)));
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel(const double* partials, int parts,
                                                            float* norm) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const float n = norm_of(partials, parts);
    if (threadIdx.x == 0) *norm = n;
}

template <typename T, int U>
__device__ __forceinline__ void scale_chunk(const Tensor& t, int64_t first, float scale) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const T* from = static_cast<const T*>(t.from) + first;
    T* to = static_cast<T*>(t.to) + first;
    const int64_t left = t.count - first;
    if (left >= kChunkBytes<U> / static_cast<int>(sizeof(T)) &&
        ((reinterpret_cast<uintptr_t>(t.from) | reinterpret_cast<uintptr_t>(t.to)) & 15u) == 0) {
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            q[u] = reinterpret_cast<const uint4*>(from)[u * kClipThreads + threadIdx.x];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[N];
            widen_piece<T>(q[u], v);
            uint4 o;
            if constexpr (sizeof(T) == 4) {
                o = make_uint4(__float_as_uint(v[0] * scale), __float_as_uint(v[1] * scale),
                               __float_as_uint(v[2] * scale), __float_as_uint(v[3] * scale));
            } else {
                o = make_uint4(pack2<T>(v[0] * scale, v[1] * scale), pack2<T>(v[2] * scale, v[3] * scale),
                               pack2<T>(v[4] * scale, v[5] * scale), pack2<T>(v[6] * scale, v[7] * scale));
            }
            reinterpret_cast<uint4*>(to)[u * kClipThreads + threadIdx.x] = o;
        }
        return;
    }
    for (int64_t at = threadIdx.x; at < left && at < kChunkBytes<U> / static_cast<int>(sizeof(T));
         at += kClipThreads)
        to[at] = from_float<T>(to_float(from[at]) * scale);
}

// Every block finds the norm from the partial sums itself (a launch less), then
// scales its chunks, the last ones first: those the squares read last, which
// L2 still holds.
template <int U>
__global__ void __launch_bounds__(kClipThreads) scale_kernel(const __grid_constant__ TensorBatch a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const float norm = norm_of(a.partials, a.parts);
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
    const float under = norm + a.eps;
    const float scale = under <= a.max_norm ? 1.0f : a.max_norm / under;   // a NaN stays one
    int n = a.tensors - 1;
    for (uint32_t i = blockIdx.x; i < a.chunks; i += gridDim.x) {
        const uint32_t c = a.chunks - 1 - i;
        while (n > 0 && c < a.at[n].chunks_before) --n;
        const Tensor& t = a.at[n];
        if (scale == 1.0f && t.to == t.from) continue;    // as it is
        const int64_t bytes = static_cast<int64_t>(c - t.chunks_before) * kChunkBytes<U>;
        if (t.dtype == TILES_BF16) scale_chunk<__nv_bfloat16, U>(t, bytes / 2, scale);
        else if (t.dtype == TILES_F16) scale_chunk<__half, U>(t, bytes / 2, scale);
        else scale_chunk<float, U>(t, bytes / 4, scale);
    }
}

// A run of tensors that one launch takes: [first, last) of the caller's, those
// without elements left out.
struct Run { int64_t first, last; };

void fill_batch(TensorBatch* b, const tiles_grad_tensor* t, Run r, int chunk_bytes) {
    b->tensors = 0;
    b->chunks = 0;
    for (int64_t i = r.first; i < r.last; ++i) {
        if (t[i].count == 0) continue;
        Tensor& e = b->at[b->tensors++];
        e.from = t[i].grad;
        e.to = t[i].out ? t[i].out : const_cast<void*>(t[i].grad);
        e.count = t[i].count;
        e.dtype = t[i].dtype;
        e.chunks_before = b->chunks;
        b->chunks += static_cast<uint32_t>((t[i].count * dtype_bytes(t[i].dtype) + chunk_bytes - 1) / chunk_bytes);
    }
}

int run_blocks(const TensorBatch& b, int sms) {
    return static_cast<int>(std::min<int64_t>(b.chunks, static_cast<int64_t>(sms) * kClipBlocksPerSm));
}

size_t clip_bytes(int64_t tensors, int sms) {
    const int64_t launches = (tensors + kTensors - 1) / kTensors;
    return kConvMinWorkspaceBytes + static_cast<size_t>(launches) * sms * kClipBlocksPerSm * 8;
}

// No output may lie over another tensor's output or gradient.
int check_apart(const tiles_grad_tensor* t, int64_t n) {
    struct Span { uintptr_t at, end; bool written; };
    try {
        std::vector<Span> spans;
        spans.reserve(static_cast<size_t>(2 * n));
        for (int64_t i = 0; i < n; ++i) {
            if (t[i].count == 0) continue;
            const uintptr_t bytes = static_cast<uintptr_t>(t[i].count) * dtype_bytes(t[i].dtype);
            const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad);
            const uintptr_t o = t[i].out ? reinterpret_cast<uintptr_t>(t[i].out) : g;
            spans.push_back({o, o + bytes, true});
            if (o != g) spans.push_back({g, g + bytes, false});
        }
        std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
        uintptr_t any = 0, written = 0;                   // ends of the spans so far
        for (const Span& s : spans) {
            if (s.at < (s.written ? any : written))
                return fail(TILES_ERR_INVALID_ARG, "two tensors overlap, and one of them is written");
            any = std::max(any, s.end);
            if (s.written) written = std::max(written, s.end);
        }
    } catch (const std::exception&) {
        return fail(TILES_ERR_TOO_LARGE, "too many tensors for the host's memory");
    }
    return TILES_OK;
}

int check_tensors(const tiles_grad_tensor* t, int64_t n, const float* norm, bool out) {
    if (n < 0 || (n && !t)) return fail(TILES_ERR_INVALID_ARG, "no tensors");
    if (n > (1 << 20)) return fail(TILES_ERR_TOO_LARGE, "more than 2^20 tensors");
    if (!norm || !element_aligned(norm, 4))
        return fail(TILES_ERR_INVALID_ARG, "norm is null or not aligned to its element");
    for (int64_t i = 0; i < n; ++i) {
        const int eb = dtype_bytes(t[i].dtype);
        if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "tensor %lld must be f16, bf16 or f32", (long long)i);
        if (t[i].count < 0) return fail(TILES_ERR_INVALID_ARG, "tensor %lld has a negative size", (long long)i);
        if (t[i].count > (int64_t(1) << 40)) return fail(TILES_ERR_TOO_LARGE, "tensor %lld exceeds 2^40", (long long)i);
        if (t[i].count == 0) continue;
        if (!t[i].grad) return fail(TILES_ERR_INVALID_ARG, "tensor %lld is null", (long long)i);
        if (!element_aligned(t[i].grad, eb) || (out && !element_aligned(t[i].out, eb)))
            return fail(TILES_ERR_MISALIGNED, "tensor %lld is not aligned to its element", (long long)i);
    }
    return TILES_OK;
}

int check_clip_workspace(void* ws, size_t ws_bytes, int64_t n, int sms) {
    const size_t need = clip_bytes(n, sms);
    if (!ws || ws_bytes < need)
        return fail(TILES_ERR_INVALID_ARG, "the norm of %lld tensors needs %zu workspace bytes", (long long)n, need);
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(TILES_ERR_MISALIGNED, "the workspace must be 16-byte aligned");
    return TILES_OK;
}

// The launches of the squares; the number of partial sums they leave.
template <int U>
int launch_squares(const tiles_grad_tensor* t, int64_t n, double* partials, int sms, int* parts, cudaStream_t st) {
    TensorBatch b{};
    *parts = 0;
    for (int64_t i = 0; i < n; i += kTensors) {
        fill_batch(&b, t, {i, std::min<int64_t>(n, i + kTensors)}, kChunkBytes<U>);
        if (b.chunks == 0) continue;
        b.partials = partials + *parts;
        const int blocks = run_blocks(b, sms);
        const int e = launch(squares_kernel<U>, dim3(blocks), dim3(kClipThreads), 0, st, b);
        if (e != cudaSuccess) return e;
        *parts += blocks;
    }
    return cudaSuccess;
}

template <int U>
int launch_clip(const tiles_grad_tensor* t, int64_t n, float max_norm, float eps, float* norm,
                double* partials, int sms, cudaStream_t st) {
    TensorBatch b{};
    int e = launch_squares<U>(t, n, partials, sms, &b.parts, st);
    if (e != cudaSuccess) return e;
    b.partials = partials;
    b.max_norm = max_norm;
    b.eps = eps;
    b.norm = norm;
    for (int64_t i = (n - 1) / kTensors * kTensors; i >= 0; i -= kTensors) {
        fill_batch(&b, t, {i, std::min<int64_t>(n, i + kTensors)}, kChunkBytes<U>);
        if (b.chunks == 0) continue;
        e = launch(scale_kernel<U>, dim3(run_blocks(b, sms)), dim3(kClipThreads), 0, st, b);
        if (e != cudaSuccess) return e;
        b.norm = nullptr;                                 // written once
    }
    if (b.norm)                                           // no elements at all
        e = launch(norm_kernel, dim3(1), dim3(kClipThreads), 0, st, static_cast<const double*>(partials), 0, norm);
    return e;
}

// Pieces a thread: small gradients are spread over more blocks.
bool few_bytes(const tiles_grad_tensor* t, int64_t n, int sms) {
    int64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) bytes += t[i].count * dtype_bytes(t[i].dtype);
    return bytes < static_cast<int64_t>(sms) * 4 * kChunkBytes<8>;
}

}  // namespace
}  // namespace tiles

using namespace tiles;

extern "C" {

size_t tiles_grad_norm_workspace_bytes(int64_t tensors) {
    if (tensors < 0 || tensors > (1 << 20)) {
        fail(TILES_ERR_INVALID_ARG, "between 0 and 2^20 tensors");
        return 0;
    }
    int sms = 0;
    if (current_sm_count(&sms) != TILES_OK) return 0;
    return clip_bytes(tensors, sms);
}

int tiles_grad_norm(const tiles_grad_tensor* t, int64_t n, float* norm, void* ws, size_t ws_bytes,
                    void* stream) {
    int s = check_tensors(t, n, norm, false), sms = 0;
    if (s != TILES_OK) return s;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    if ((s = check_clip_workspace(ws, ws_bytes, n, sms)) != TILES_OK) return s;
    double* partials = reinterpret_cast<double*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int parts = 0;
    int e = few_bytes(t, n, sms) ? launch_squares<2>(t, n, partials, sms, &parts, st)
                                 : launch_squares<8>(t, n, partials, sms, &parts, st);
    if (e == cudaSuccess)
        e = launch(norm_kernel, dim3(1), dim3(kClipThreads), 0, st, static_cast<const double*>(partials), parts, norm);
    return launch_status(e, "gradient norm");
}

int tiles_clip_grads(const tiles_grad_tensor* t, int64_t n, float max_norm, float eps, float* norm,
                     void* ws, size_t ws_bytes, void* stream) {
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f))
        return fail(TILES_ERR_INVALID_ARG, "max_norm and eps must be >= 0");
    int s = check_tensors(t, n, norm, true), sms = 0;
    if (s != TILES_OK) return s;
    if ((s = check_apart(t, n)) != TILES_OK) return s;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    if ((s = check_clip_workspace(ws, ws_bytes, n, sms)) != TILES_OK) return s;
    double* partials = reinterpret_cast<double*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int e = few_bytes(t, n, sms) ? launch_clip<2>(t, n, max_norm, eps, norm, partials, sms, st)
                                       : launch_clip<8>(t, n, max_norm, eps, norm, partials, sms, st);
    return launch_status(e, "gradient clipping");
}

}  // extern "C"

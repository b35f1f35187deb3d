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

// Tensors a launch takes: their descriptions travel with it as arguments (at most
// 32,764 bytes), so that nothing on the host has to outlive the call and a captured
// launch carries them.  Three sizes, as the host copies all of it: 600 tensors of
// 20,000 bf16 in one launch of the squares and one of the scaling 17 us, in five of each
// 37 (both in a graph, with nothing else between them).
constexpr int kTensors = 1000, kSomeTensors = 120, kFewTensors = 16;
constexpr int kClipThreads = 256;
constexpr int kMostBlocksPerSm = 8;

struct Tensor {
    const void* from;
    void* to;
    int64_t count;
};

// A sum of squares: that of the elements whose squares fp32 holds, and of others.
struct alignas(16) Partial {
    float near;
    double far;

    // (Without an fp64 comparison.)
    __device__ __forceinline__ bool has_far() const { return __double_as_longlong(far) != 0; }
};

template <int N>
struct TensorBatch {
    int32_t tensors;
    uint32_t chunks;
    int32_t parts;                             // partial sums of all launches; -1: norm is there
    float max_norm, eps;
    uint32_t once;                             // chunks before this one are not read again soon
    Partial* partials;                         // this launch's first, or (scaling) the very first
    float* norm;
    uint32_t chunks_before[N];                 // of the launch's tensors before each
    uint8_t dtype[N];
    Tensor at[N];
};
static_assert(sizeof(TensorBatch<kTensors>) <= 32764, "arguments of one launch");

// A tensor is seen as 16-byte pieces that start on 16 bytes, of which its first
// and last may hold other memory too; U pieces a thread are a chunk, what a
// block takes at a time.
template <int U> constexpr int kChunkPieces = U * kClipThreads;

__host__ __device__ __forceinline__ int misaligned(const void* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
}

template <typename T>
__device__ __forceinline__ void widen_piece(const uint4& q, float (&v)[16 / sizeof(T)]) {
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

// The tensor that chunk c is of: the last one that starts at c or before.
template <int N>
__device__ __forceinline__ int tensor_of(const TensorBatch<N>& a, uint32_t c) {
    int lo = 0, n = a.tensors;
    while (n > 1) {
        const int half = n / 2;
        if (a.chunks_before[lo + half] <= c) lo += half;
        n -= half;
    }
    return lo;
}

// The 16 bytes from byte `at` of a tensor on, those outside it as zeros, element
// by element.
template <typename T>
__device__ __forceinline__ uint4 partial_piece(const T* from, int64_t at, int64_t count) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const int64_t first = at / static_cast<int64_t>(sizeof(T));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (first + i < 0 || first + i >= count) continue;
        if constexpr (sizeof(T) == 4)
            w[i] = reinterpret_cast<const uint32_t*>(from)[first + i];
        else
            w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(from)[first + i]) << 16 * (i & 1);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Squares and their sums are fp32: a thread adds its pieces of a chunk in four
// chains, its chunks' sums with what their additions round off, and the threads'
// sums in a tree.  (fp64 takes this chip 64 times as long: with sums in fp64
// from a chunk's on 5 million bf16 elements took 13.8 us to clip, not 10.6.)  A chunk's
// share that leaves fp32's range (over 2^80, so that no sum of such leaves it
// either, or under 2^-90 and not of zeros alone) the thread takes once more, in fp64,
// and that sum stays apart.
constexpr float kSmallSquares = 0x1p-90f, kBigSquares = 0x1p80f;

struct Sum {
    float s = 0.0f, lost = 0.0f;               // lost: what the additions rounded off
    double far = 0.0;
    bool has_far = false;

    __device__ __forceinline__ void add(float x) {
        const float t = s + x, b = t - s;
        lost += (s - (t - b)) + (x - b);
        s = t;
    }
    __device__ __forceinline__ void add_far(double x) {
        far += x;
        has_far = true;
    }
};

template <typename T> __device__ __forceinline__ constexpr uint32_t magnitude_bits() {
    return sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
}

template <typename T, int U>
__device__ __noinline__ double squares_in_double(const Tensor& t, int64_t first) {
    double s = 0.0;
    for (int u = 0; u < U; ++u) {
        const int64_t at = (first + u * kClipThreads + threadIdx.x) * 16 - misaligned(t.from);
        if (at >= t.count * static_cast<int64_t>(sizeof(T))) break;
        float v[16 / sizeof(T)];
        widen_piece<T>(partial_piece(static_cast<const T*>(t.from), at, t.count), v);
        for (float e : v) s += static_cast<double>(e) * static_cast<double>(e);
    }
    return s;
}

// A load of what L2 need not keep.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
    uint64_t policy;
    uint4 v;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}

// The squares of a thread's share of the chunk that starts at piece `first`, to its sum.
template <typename T, int U>
__device__ __forceinline__ void chunk_squares(const Tensor& t, int64_t first, bool once, Sum& sum) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const T* from = static_cast<const T*>(t.from);
    const int64_t bytes = t.count * static_cast<int64_t>(sizeof(T));
    const int64_t start = first * 16 - misaligned(from);       // the chunk's first byte in the tensor
    const char* at = static_cast<const char*>(t.from) + start;
    uint4 q[U];
    if (start >= 0 && start + kChunkPieces<U> * 16 <= bytes) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint4* p = reinterpret_cast<const uint4*>(at) + u * kClipThreads + threadIdx.x;
            q[u] = once ? load_once(p) : *p;
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t b = start + (u * kClipThreads + static_cast<int>(threadIdx.x)) * 16;
            q[u] = make_uint4(0, 0, 0, 0);
            if (b >= 0 && b + 16 <= bytes)
                q[u] = reinterpret_cast<const uint4*>(at)[u * kClipThreads + threadIdx.x];
            else if (b < bytes)
                q[u] = partial_piece(from, b, t.count);
        }
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        any |= q[u].x | q[u].y | q[u].z | q[u].w;
        float v[N];
        widen_piece<T>(q[u], v);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
    }
    const float all = (s[0] + s[1]) + (s[2] + s[3]);
    if (!(all >= kSmallSquares && all <= kBigSquares) && (any & magnitude_bits<T>()))
        sum.add_far(squares_in_double<T, U>(t, first));
    else
        sum.add(all);
}

// The sum over a block; every thread gets it.  Both parts, the far one where any
// thread has one.
__device__ __forceinline__ Partial block_sum(const Sum& sum) {
    constexpr uint32_t kAll = 0xffffffffu;
    __shared__ float near[kClipThreads / 32];
    __shared__ double far[kClipThreads / 32];
    const int warp = threadIdx.x >> 5;
    float s = sum.s + sum.lost;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kAll, s, d);
    if ((threadIdx.x & 31) == 0) near[warp] = s;
    Partial p{0.0f, 0.0};
    if (__syncthreads_or(sum.has_far)) {
        double f = sum.far;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) f += __shfl_xor_sync(kAll, f, d);
        if ((threadIdx.x & 31) == 0) far[warp] = f;
        __syncthreads();
        for (double w : far) p.far += w;
    }
#pragma unroll
    for (float w : near) p.near += w;
    return p;
}

// One partial sum a block, over the chunks blockIdx.x, + gridDim.x, ...  256
// million bf16 elements 78 us with the norm: 98% of the measured copy bandwidth.
template <int U, int N>
__global__ void __launch_bounds__(kClipThreads, U > 4 ? 4 : 8)
    squares_kernel(const __grid_constant__ TensorBatch<N> a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    Sum s;
    for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const int n = tensor_of(a, c);
        const Tensor& t = a.at[n];
        const int64_t first = static_cast<int64_t>(c - a.chunks_before[n]) * kChunkPieces<U>;
        if (a.dtype[n] == TILES_BF16) chunk_squares<__nv_bfloat16, U>(t, first, c < a.once, s);
        else if (a.dtype[n] == TILES_F16) chunk_squares<__half, U>(t, first, c < a.once, s);
        else chunk_squares<float, U>(t, first, c < a.once, s);
    }
    const Partial p = block_sum(s);
    if (threadIdx.x == 0) a.partials[blockIdx.x] = p;
}

// The square root of a sum of squares.  fp64's takes this chip a microsecond.
__device__ __forceinline__ float root_of(const Partial& p) {
    return !p.has_far() ? sqrtf(p.near) : static_cast<float>(sqrt(static_cast<double>(p.near) + p.far));
}

// The norm from all partial sums, in a fixed order (every thread of a block
// gets it).
__device__ __forceinline__ float norm_of(const Partial* partials, int parts) {
    Sum s;
#pragma unroll 2
    for (int i = threadIdx.x; i < parts; i += kClipThreads) {
        const Partial p = partials[i];
        s.add(p.near);
        if (p.has_far()) s.add_far(p.far);
    }
    return root_of(block_sum(s));
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel(const Partial* partials, int parts,
                                                            float* norm) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const float n = norm_of(partials, parts);
    if (threadIdx.x == 0) *norm = n;
}

__device__ __forceinline__ float factor_of(float norm, float max_norm, float eps) {
    const float under = norm + eps;
    return under <= max_norm ? 1.0f : max_norm / under;        // a NaN stays one
}

template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4& q, float scale) {
    float v[16 / sizeof(T)];
    widen_piece<T>(q, v);
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(v[0] * scale), __float_as_uint(v[1] * scale),
                          __float_as_uint(v[2] * scale), __float_as_uint(v[3] * scale));
    else
        return make_uint4(pack2<T>(v[0] * scale, v[1] * scale), pack2<T>(v[2] * scale, v[3] * scale),
                          pack2<T>(v[4] * scale, v[5] * scale), pack2<T>(v[6] * scale, v[7] * scale));
}

// The piece of what is written that starts at byte b: the elements of it that
// are the tensor's, one by one where it holds others too.
template <typename T>
__device__ __forceinline__ void scale_piece(const Tensor& t, int64_t b, float scale) {
    const int64_t bytes = t.count * static_cast<int64_t>(sizeof(T));
    const char* from = static_cast<const char*>(t.from);
    if (b >= 0 && b + 16 <= bytes) {
        const uint4 q = unaligned16(from + b, Extent{from, from + bytes}, sizeof(T));
        *reinterpret_cast<uint4*>(static_cast<char*>(t.to) + b) = scaled<T>(q, scale);
        return;
    }
    const int64_t first = b / static_cast<int64_t>(sizeof(T));
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = first + i >= 0 && first + i < t.count ? to_float(static_cast<const T*>(t.from)[first + i]) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (first + i >= 0 && first + i < t.count)
            static_cast<T*>(t.to)[first + i] = from_float<T>(v[i] * scale);
}

// Finds the norm, from the partial sums itself (a launch less) or where
// norm_kernel left it (parts < 0), then scales its chunks, the last ones first:
// those the squares read last, which L2 still holds.  256 million bf16 elements, norm and scaling:
// 228 us, 1.54 GB at the measured copy bandwidth.
template <int U, int N>
__global__ void __launch_bounds__(kClipThreads, U > 4 ? 4 : 8)
    scale_kernel(const __grid_constant__ TensorBatch<N> a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float scale = 0.0f;
    bool known = false;
    for (uint32_t i = blockIdx.x; i < a.chunks; i += gridDim.x) {
        const uint32_t c = a.chunks - 1 - i;
        const int n = tensor_of(a, c);
        const Tensor& t = a.at[n];
        // In pieces of what is written.
        constexpr int kStep = kClipThreads * 16;
        const int64_t bytes = t.count * (a.dtype[n] == TILES_F32 ? 4 : 2);
        const int64_t at = static_cast<int64_t>(c - a.chunks_before[n]) * (U * kStep) - misaligned(t.to);
        const int64_t mine = at + static_cast<int>(threadIdx.x) * 16;
        const bool whole = misaligned(t.from) == misaligned(t.to) && at >= 0 && at + U * kStep <= bytes;
        uint4 q[U];
        if (whole)
#pragma unroll
            for (int u = 0; u < U; ++u)
                q[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(t.from) + mine + u * kStep);
        if (!known) {                                     // (with the first chunk on its way)
            const float norm = a.parts < 0 ? *a.norm : norm_of(a.partials, a.parts);
            if (a.parts >= 0 && a.norm && i == 0 && threadIdx.x == 0) *a.norm = norm;
            scale = factor_of(norm, a.max_norm, a.eps);
            known = true;
        }
        if (scale == 1.0f && t.to == t.from) continue;    // as it is
        auto write = [&](auto zero) {
            using T = decltype(zero);
            if (whole) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    *reinterpret_cast<uint4*>(static_cast<char*>(t.to) + mine + u * kStep) = scaled<T>(q[u], scale);
            } else {
#pragma unroll 1
                for (int64_t b = mine, end = min(bytes, mine + U * kStep); b < end; b += kStep)
                    scale_piece<T>(t, b, scale);
            }
        };
        if (a.dtype[n] == TILES_BF16) write(__nv_bfloat16());
        else if (a.dtype[n] == TILES_F16) write(__half());
        else write(float());
    }
}

// A run of tensors that one launch takes: [first, last) of the caller's, those
// without elements left out.
struct Run { int64_t first, last; };

// `written`: in pieces of what is written, not of what is read.
template <int N>
void fill_batch(TensorBatch<N>* b, const tiles_grad_tensor* t, Run r, int chunk_pieces, bool written) {
    b->tensors = 0;
    b->chunks = 0;
    const int64_t chunk = static_cast<int64_t>(chunk_pieces) * 16;
    for (int64_t i = r.first; i < r.last; ++i) {
        if (t[i].count == 0) continue;
        const int n = b->tensors++;
        Tensor& e = b->at[n];
        e.from = t[i].grad;
        e.to = t[i].out ? t[i].out : const_cast<void*>(t[i].grad);
        e.count = t[i].count;
        b->dtype[n] = static_cast<uint8_t>(t[i].dtype);
        b->chunks_before[n] = b->chunks;
        const int64_t bytes = t[i].count * dtype_bytes(t[i].dtype) + misaligned(written ? e.to : e.from);
        b->chunks += static_cast<uint32_t>((bytes + chunk - 1) / chunk);
    }
}

template <int U> constexpr int kBlocksPerSm = U > 4 ? 4 : 8;

template <int U, int N>
int run_blocks(const TensorBatch<N>& b, int sms) {
    return static_cast<int>(std::min<int64_t>(b.chunks, static_cast<int64_t>(sms) * kBlocksPerSm<U>));
}

size_t clip_bytes(int64_t tensors, int sms) {
    const int64_t launches = (tensors + kTensors - 1) / kTensors;
    return kConvMinWorkspaceBytes + static_cast<size_t>(launches) * sms * kMostBlocksPerSm * sizeof(Partial);
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
    int64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) {
        const int eb = dtype_bytes(t[i].dtype);
        if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "tensor %lld must be f16, bf16 or f32", (long long)i);
        if (t[i].count < 0) return fail(TILES_ERR_INVALID_ARG, "tensor %lld has a negative size", (long long)i);
        if (t[i].count > (int64_t(1) << 40)) return fail(TILES_ERR_TOO_LARGE, "tensor %lld exceeds 2^40", (long long)i);
        if (t[i].count == 0) continue;
        bytes += t[i].count * eb;
        if (bytes > (int64_t(1) << 46)) return fail(TILES_ERR_TOO_LARGE, "the gradients exceed 2^46 bytes");
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

int64_t total_bytes(const tiles_grad_tensor* t, int64_t n) {
    int64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) bytes += t[i].count * dtype_bytes(t[i].dtype);
    return bytes;
}

// What L2 (129 MB) is asked to keep of the gradients for the scaling, which
// starts with what was read last: 256 million bf16 elements 228 us against 236.
constexpr int64_t kKeptBytes = 100000000;

// The launches of the squares; the number of partial sums they leave.  `again`:
// the gradients are read again.
template <int U, int N>
int launch_squares(const tiles_grad_tensor* t, int64_t n, bool again, Partial* partials, int sms, int* parts,
                   cudaStream_t st) {
    TensorBatch<N> b;                                     // (its arrays need no zeros)
    *parts = 0;
    constexpr int64_t kChunk = kChunkPieces<U> * 16;
    int64_t left = again ? total_bytes(t, n) : 0;
    for (int64_t i = 0; i < n; i += N) {
        fill_batch(&b, t, {i, std::min<int64_t>(n, i + N)}, kChunkPieces<U>, false);
        if (b.chunks == 0) continue;
        b.partials = partials + *parts;
        b.once = static_cast<uint32_t>(
            std::min<int64_t>(b.chunks, std::max<int64_t>(0, left - kKeptBytes) / kChunk));
        left -= b.chunks * kChunk;
        const int blocks = run_blocks<U>(b, sms);
        const int e = launch(squares_kernel<U, N>, dim3(blocks), dim3(kClipThreads), 0, st, b);
        if (e != cudaSuccess) return e;
        *parts += blocks;
    }
    return cudaSuccess;
}

template <int U, int N>
int launch_clip(const tiles_grad_tensor* t, int64_t n, float max_norm, float eps, float* norm,
                Partial* partials, int sms, cudaStream_t st) {
    TensorBatch<N> b;
    int e = launch_squares<U, N>(t, n, true, partials, sms, &b.parts, st);
    if (e != cudaSuccess) return e;
    b.partials = partials;
    b.max_norm = max_norm;
    b.eps = eps;
    b.norm = norm;
    // One launch's partial sums every block of the scaling adds up itself; where there
    // are more one block makes the norm first (of 17 launches 131 us against 163).
    if (b.parts > kMostBlocksPerSm * sms) {
        e = launch(norm_kernel, dim3(1), dim3(kClipThreads), 0, st, static_cast<const Partial*>(partials), b.parts,
                   norm);
        if (e != cudaSuccess) return e;
        b.parts = -1;
    }
    for (int64_t i = (n - 1) / N * N; i >= 0; i -= N) {
        fill_batch(&b, t, {i, std::min<int64_t>(n, i + N)}, kChunkPieces<U>, true);
        if (b.chunks == 0) continue;
        e = launch(scale_kernel<U, N>, dim3(std::min<uint32_t>(b.chunks, 1u << 30)), dim3(kClipThreads), 0, st, b);
        if (e != cudaSuccess) return e;
        if (b.parts >= 0) b.norm = nullptr;               // written once
    }
    if (b.parts == 0)                                     // no elements at all
        e = launch(norm_kernel, dim3(1), dim3(kClipThreads), 0, st, static_cast<const Partial*>(partials), 0, norm);
    return e;
}

// Pieces a thread: small gradients are spread over more blocks.
bool few_bytes(const tiles_grad_tensor* t, int64_t n, int sms) {
    return total_bytes(t, n) < static_cast<int64_t>(sms) * 4 * kChunkPieces<8> * 16;
}

// The instance for few or many bytes, and for so many tensors.
template <typename F>
F pick(bool few, int64_t n, const F (&some)[3], const F (&much)[3]) {
    const int i = n <= kFewTensors ? 0 : n <= kSomeTensors ? 1 : 2;
    return few ? some[i] : much[i];
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
    Partial* partials = reinterpret_cast<Partial*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int parts = 0;
    const auto squares =
        pick<decltype(&launch_squares<2, kTensors>)>(
            few_bytes(t, n, sms), n,
            {launch_squares<2, kFewTensors>, launch_squares<2, kSomeTensors>, launch_squares<2, kTensors>},
            {launch_squares<8, kFewTensors>, launch_squares<8, kSomeTensors>, launch_squares<8, kTensors>});
    int e = squares(t, n, false, partials, sms, &parts, st);
    if (e == cudaSuccess)
        e = launch(norm_kernel, dim3(1), dim3(kClipThreads), 0, st, static_cast<const Partial*>(partials), parts, norm);
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
    Partial* partials = reinterpret_cast<Partial*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto clip =
        pick<decltype(&launch_clip<2, kTensors>)>(
            few_bytes(t, n, sms), n,
            {launch_clip<2, kFewTensors>, launch_clip<2, kSomeTensors>, launch_clip<2, kTensors>},
            {launch_clip<8, kFewTensors>, launch_clip<8, kSomeTensors>, launch_clip<8, kTensors>});
    const int e = clip(t, n, max_norm, eps, norm, partials, sms, st);
    return launch_status(e, "gradient clipping");
}

}  // extern "C"

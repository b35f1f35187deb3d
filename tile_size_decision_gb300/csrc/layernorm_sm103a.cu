// Layer norm with the residual's addition (16-bit, fp32 or scaled 8-bit
// output) and its gradients.
//
// As the root-mean-square norm, both read and write every element once: DRAM
// bounds them, if the instructions do not, of which there are more (the mean
// comes first, then what is left after it).  So the arithmetic is done on pairs
// of fp32, and several sums of a row go through its lanes together.
//
// A row's elements are taken about a mean m in fp32, d = h - m; the sums of d
// and d^2 give what m was off by, off = mean(d), and var = mean(d^2) - off^2: a
// row whose mean is far larger than its spread loses nothing (without off the
// error of m, up to 2^-20 |m|, would shift all of y).
#include "row_ops.cuh"

namespace tiles {
namespace {

// Eight columns as four pairs.
struct Eight {
    uint64_t p[4];

    __device__ __forceinline__ void fill(float v) {
        const uint64_t q = ptx::pair(v, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = q;
    }
    __device__ __forceinline__ void from(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ptx::pair(v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ void to(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = ptx::unpair(p[i]);
            v[2 * i] = t.x;
            v[2 * i + 1] = t.y;
        }
    }
    // The sum of all eight.
    __device__ __forceinline__ float sum() const {
        const float2 t = ptx::unpair(ptx::add2(ptx::add2(p[0], p[1]), ptx::add2(p[2], p[3])));
        return t.x + t.y;
    }
};

// Where the columns are all inside the row (VEC: eight together), v; else zeros
// for those past its end.
template <bool VEC>
__device__ __forceinline__ void keep(Eight& v, int c, int cols) {
    if constexpr (VEC) {
        if (c >= cols) v.fill(0.0f);
    } else {
        if ((c | 127) < cols) return;
        float t[8];
        v.to(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = column<false>(c, i) < cols ? t[i] : 0.0f;
        v.from(t);
    }
}

// Sums of USED values over the threads of one row (blockDim.x of them, whole
// warps, at most W); every thread gets them.  N is the power of two over USED:
// five values take 8 shuffles in a warp (not 25) and 7 among the warps.  `slot`
// holds W N floats; between two uses of the same the row's threads meet at a
// barrier.  RING: the row's own barrier, and slots that hold zeros where the row
// has fewer warps (kernels of one row a block would pay for that each time).
template <int N, int USED, int W, bool RING>
__device__ __forceinline__ void row_sums(float (&s)[N], float* slot) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    float x = fold<N, USED>(s);
    if (blockDim.x > 32) {
        const int values = (blockDim.x >> 5) * N;
        if (lane < N) slot[(threadIdx.x >> 5) * N + lane] = x;
        if constexpr (RING) ptx::named_barrier(1 + threadIdx.y, blockDim.x);
        else __syncthreads();
        x = lane < (RING ? W * N : values) ? slot[lane] : 0.0f;
#pragma unroll
        for (int i = 32; i < W * N; i *= 2)
            if (values > i)
#pragma unroll
                for (int k = i; k < 2 * i; k += 32)
                    x += RING || lane + k < values ? slot[lane + k] : 0.0f;
#pragma unroll
        for (int d = 16; d >= N; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
    }
    if constexpr (N == 1) {
        s[0] = x;
    } else {
#pragma unroll
        for (int j = 0; j < USED; ++j) s[j] = __shfl_sync(kAll, x, j);
    }
}

// Zeros in the slots, by all threads of the block, before their first use (which
// comes after a barrier).
__device__ __forceinline__ void clear_slots(float* slots, int n) {
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < n; i += blockDim.x * blockDim.y)
        slots[i] = 0.0f;
    __syncthreads();
}

// (var + eps)^(-1/2) from the mean of d^2 and of d.  The variance is no less
// than 0, whatever the two roundings leave; a NaN stays one, and squares whose sum
// leaves fp32's range make one: the root of an infinity would be 0 and y the bias.
__device__ __forceinline__ float inverse_root(float square, float off, float eps) {
    const float var = fmaf(square, 0.0f, square - off * off);
    return rsqrtf((var < 0.0f ? 0.0f : var) + eps);
}

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

// d times rstd, times w plus b, to y: `shift` is -off rstd.  All lanes of the
// 16 that hold a block of 128 columns come here together.
template <typename T, bool VEC, bool FP8>
__device__ __forceinline__ void emit(const LayerArgs& a, int64_t row, int c, int cols, const Eight& d,
                                     uint64_t rstd, uint64_t shift, const Eight& w, const Eight& b) {
    Eight y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y.p[i] = ptx::fma2(ptx::fma2(d.p[i], rstd, shift), w.p[i], b.p[i]);
    if constexpr (FP8) {
        // What lies past the row's end must not reach the short last block's
        // scale (it may be a NaN by now).
        keep<VEC>(y, c, cols);
        float v[8];
        y.to(v);
        const float s = max_nan(__fdiv_rn(block_amax(amax8(v)), kE4m3Max), kTinyScale), inv = __frcp_rn(s);
        const uint64_t inv2 = ptx::pair(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) y.p[i] = ptx::mul2(y.p[i], inv2);
        y.to(v);
        store8_e4m3<VEC>(static_cast<uint8_t*>(a.y) + row * a.ldy, c, cols, v);
        if ((threadIdx.x & 15) == 0 && c < cols)
            a.scales[row * a.scale_row + c / kBlock * a.scale_block] = s;
    } else {
        float v[8];
        y.to(v);
        store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy, c, cols, v);
    }
}

template <bool VEC>
__device__ __forceinline__ void load_affine(const LayerArgs& a, int c, int cols, Eight& w, Eight& b) {
    float t[8];
    load8_any<VEC>(a.weight, a.weight_dtype, c, cols, t);
    w.from(t);
    b.fill(0.0f);
    if (a.bias) {
        load8_any<VEC>(a.bias, a.weight_dtype, c, cols, t);
        b.from(t);
    }
}

// One row per blockDim.x threads, blockDim.y rows per block; the layout of
// vectors over threads is the root-mean-square norm's.  VPT == 0 takes rows of
// any length: it reads h again from x and the residual for the variance and
// for the output.
template <typename T, int VPT, bool VEC, bool FP8>
__global__ void __launch_bounds__(kMaxThreads, VPT == 1 && VEC ? 2 : 1)
    layernorm_kernel(const LayerArgs a) {
    __shared__ float slots[32 + 64];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;                    // whole warps: blockDim.y > 1 only with 32 threads a row
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.0f / static_cast<float>(cols);
    auto load_h = [&](int c, Eight& v) {
        float t[8];
        load8<T, VEC>(x, c, cols, t);
        v.from(t);
        if (r) {
            load8<T, VEC>(r, c, cols, t);
            Eight q;
            q.from(t);
#pragma unroll
            for (int i = 0; i < 4; ++i) v.p[i] = ptx::add2(v.p[i], q.p[i]);
        }
    };
    auto store_h = [&](int c, const Eight& v) {
        if (!h) return;
        float t[8];
        v.to(t);
        store8<T, VEC>(h, c, cols, t);
    };
    // d = v - mean (zeros past the row's end); its sums are added to sq.
    float sum[1] = {0.0f}, sq[2] = {0.0f, 0.0f};
    auto centre = [&](int c, Eight& v, float mean) {
        const uint64_t less = ptx::pair(-mean, -mean);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = ptx::add2(v.p[i], less);
        keep<VEC>(v, c, cols);
    };
    auto squares = [&](const Eight& v) {
        Eight q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q.p[i] = ptx::mul2(v.p[i], v.p[i]);
        sq[0] += v.sum();
        sq[1] += q.sum();
    };
    const int step = blockDim.x * 8, tid = threadIdx.x;
    Eight w, b;
    if constexpr (VPT > 0) {
        Eight v[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) load_h(j * step + tid * 8, v[j]);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            store_h(j * step + tid * 8, v[j]);
            sum[0] += v[j].sum();
        }
        row_sums<1, 1, 32, false>(sum, slots);
        const float mean = sum[0] * inv_n;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            centre(j * step + tid * 8, v[j], mean);
            squares(v[j]);
        }
        row_sums<2, 2, 32, false>(sq, slots + 32);
        const float off = sq[0] * inv_n, rstd = inverse_root(sq[1] * inv_n, off, a.eps);
        const uint64_t rstd2 = ptx::pair(rstd, rstd), shift = ptx::pair(-off * rstd, -off * rstd);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * step + tid * 8;
            load_affine<VEC>(a, c, cols, w, b);
            emit<T, VEC, FP8>(a, row, c, cols, v[j], rstd2, shift, w, b);
        }
    } else {
        Eight v;
        for (int c0 = 0; c0 < cols; c0 += step) {
            load_h(c0 + tid * 8, v);
            sum[0] += v.sum();
        }
        row_sums<1, 1, 32, false>(sum, slots);
        const float mean = sum[0] * inv_n;
        for (int c0 = 0; c0 < cols; c0 += step) {
            load_h(c0 + tid * 8, v);
            centre(c0 + tid * 8, v, mean);
            squares(v);
        }
        row_sums<2, 2, 32, false>(sq, slots + 32);
        const float off = sq[0] * inv_n, rstd = inverse_root(sq[1] * inv_n, off, a.eps);
        const uint64_t rstd2 = ptx::pair(rstd, rstd), shift = ptx::pair(-off * rstd, -off * rstd);
        for (int c0 = 0; c0 < cols; c0 += step) {
            const int c = c0 + tid * 8;
            load_h(c, v);
            // h may be stored over x or the residual: after its own read.
            store_h(c, v);
            centre(c, v, mean);
            load_affine<VEC>(a, c, cols, w, b);
            emit<T, VEC, FP8>(a, row, c, cols, v, rstd2, shift, w, b);
        }
    }
}

// ---- rows on their way in ---------------------------------------------------------
//
// As the root-mean-square norm's ring, for one block of up to kRows threads an
// SM, blockDim.x of them a row: the pitch of the ring is a constant, the
// addresses of a thread's rows are kept and advanced, and what lies past a row's
// end is zeroed once and never copied, so that reads ask nothing.  (These
// kernels are near their instructions' limit.)
constexpr int kRows = 512;
constexpr int kStages = 3;

template <typename T, int N, int VPT>
struct Ring {
    static constexpr int PIECES = static_cast<int>(sizeof(T)) / 2;   // 16-byte pieces of a vector
    static constexpr int STAGE = N * VPT * PIECES * kRows;           // pieces a stage
    static constexpr size_t BYTES = static_cast<size_t>(kStages) * STAGE * 16;

    uint4* at;
    bool in[VPT];                              // whether the thread's vector lies in the row

    __device__ __forceinline__ Ring(uint4* smem, int step, int cols) {
        at = smem + threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            in[j] = j * step + static_cast<int>(threadIdx.x) * 8 < cols;
            if (in[j]) continue;
            for (int s = 0; s < kStages; ++s)
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int p = 0; p < PIECES; ++p)
                        at[s * STAGE + ((n * VPT + j) * PIECES + p) * kRows] = make_uint4(0, 0, 0, 0);
        }
    }
    // Start the copies of matrix n's vectors (from its first one) into `stage`.
    __device__ __forceinline__ void copy(int stage, int n, const T* from, int step) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (in[j])
#pragma unroll
                for (int p = 0; p < PIECES; ++p)
                    ptx::cp_async_16(at + stage * STAGE + ((n * VPT + j) * PIECES + p) * kRows,
                                     reinterpret_cast<const uint4*>(from + j * step) + p);
    }
    __device__ __forceinline__ void read(int stage, int n, int j, Eight& v) const {
        uint4 q[PIECES];
#pragma unroll
        for (int p = 0; p < PIECES; ++p) q[p] = at[stage * STAGE + ((n * VPT + j) * PIECES + p) * kRows];
        float t[8];
        widen8<T>(q, t);
        v.from(t);
    }
};

// The same with the rows' pieces 16-byte aligned: one block an SM, blockDim.y
// rows at a time (their threads meet at barriers of their own), the next two on
// their way in.  The sums of one row go together with the mean of the next, so
// that a row costs one barrier.  16384 x 4096 bf16 rows with residual 83.3 us,
// 96% of the measured copy bandwidth; one row at a time without the ring 110.
template <typename T, int VPT, bool FP8, bool RES>
__global__ void __launch_bounds__(kRows)
    layernorm_ring_kernel(const LayerArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[8][2][16 * 4];          // rows of several warps: at most 8
    float(*const mine)[16 * 4] = slots[blockDim.x > 32 ? threadIdx.y : 0];
    clear_slots(&slots[0][0][0], sizeof(slots) / 4);
    const int step = blockDim.x * 8, tid = threadIdx.x, cols = static_cast<int>(a.cols);
    Ring<T, RES ? 2 : 1, VPT> ring(ring_smem, step, cols);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y, ahead = row;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx + tid * 8;
    const T* r = RES ? static_cast<const T*>(a.residual) + row * a.ldr + tid * 8 : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
    auto fetch = [&](int stage) {
        if (ahead < a.rows) {
            ring.copy(stage, 0, x, step);
            if constexpr (RES) ring.copy(stage, 1, r, step);
        }
        ptx::cp_async_commit();
        ahead += stride;
        x += stride * a.ldx;
        if constexpr (RES) r += stride * a.ldr;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    Eight w[VPT], b[VPT], v[VPT];
    float mask[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        load_affine<true>(a, j * step + tid * 8, cols, w[j], b[j]);
        mask[j] = ring.in[j] ? -1.0f / static_cast<float>(cols) : 0.0f;
    }
    const float inv_n = 1.0f / static_cast<float>(cols);
    // h of a row that has arrived, in v; stored; its sum.
    auto take = [&](int stage) {
        Eight all;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            ring.read(stage, 0, j, v[j]);
            if constexpr (RES) {
                Eight q;
                ring.read(stage, 1, j, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j].p[i] = ptx::add2(v[j].p[i], q.p[i]);
            }
            if (h) {
                float t[8];
                v[j].to(t);
                store8<T, true>(h, j * step + tid * 8, cols, t);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) all.p[i] = j ? ptx::add2(all.p[i], v[j].p[i]) : v[j].p[i];
        }
        if (h) h += stride * a.ldh;
        return all.sum();
    };
    ptx::cp_async_wait_groups<kStages - 2>();
    float s[4];
    s[0] = row < a.rows ? take(0) : 0.0f;
    row_sums<4, 1, 16, true>(s, mine[1]);
    float total = s[0];
    int stage = 0, turn = 0;
    for (; row < a.rows; row += stride, turn ^= 1) {
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        Eight d[VPT], d1, d2;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const uint64_t less = ptx::pair(total * mask[j], total * mask[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[j].p[i] = ptx::add2(v[j].p[i], less);
                d1.p[i] = j ? ptx::add2(d1.p[i], d[j].p[i]) : d[j].p[i];
                d2.p[i] = j ? ptx::fma2(d[j].p[i], d[j].p[i], d2.p[i]) : ptx::mul2(d[j].p[i], d[j].p[i]);
            }
        }
        s[0] = d1.sum();
        s[1] = d2.sum();
        s[2] = 0.0f;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        ptx::cp_async_wait_groups<kStages - 2>();
        if (row + stride < a.rows) s[2] = take(stage);
        row_sums<4, 3, 16, true>(s, mine[turn]);
        total = s[2];
        const float off = s[0] * inv_n, rstd = inverse_root(s[1] * inv_n, off, a.eps);
        const uint64_t rstd2 = ptx::pair(rstd, rstd), shift = ptx::pair(-off * rstd, -off * rstd);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            emit<T, true, FP8>(a, row, j * step + tid * 8, cols, d[j], rstd2, shift, w[j], b[j]);
    }
}

// ---- rows that start anywhere, on their way in ------------------------------------
//
// Such a row (of 16-bit elements) comes in as the 16-byte pieces of memory that hold
// it, and its threads read their columns out of what all of them have copied.  So a thread waits for a row's copies before the barrier
// that the row before it has anyway, and what was read before a barrier makes
// room after it.

// A thread's vector c of such a row: four pairs of neighbouring columns, those of a
// warp side by side (64 columns), 256 columns a warp.
__device__ __forceinline__ int pair_column(int c, int k) { return (c & ~255) + ((c >> 3) & 31) * 2 + 64 * k; }

// Out of shared memory, where 4 more bytes may be read behind a row; columns past its
// end read as zero.
__device__ __forceinline__ void load_words(const char* row, int c, int cols, uint32_t (&w)[4]) {
    const uint32_t* at = reinterpret_cast<const uint32_t*>(row - (reinterpret_cast<uintptr_t>(row) & 2u)) +
                         pair_column(c, 0) / 2;
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 2u) * 8;
    if ((c | 255) < cols) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(at[32 * k], at[32 * k + 1], shift);
    } else {
        const int left = cols - pair_column(c, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = left > 64 * k
                       ? __funnelshift_r(at[32 * k], at[32 * k + 1], shift) & (left > 64 * k + 1 ? ~0u : 0xffffu)
                       : 0u;
    }
}

template <typename T>
__device__ __forceinline__ void widen_words(const uint32_t (&w)[4], Eight& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = unpack2<T>(w[k]);
        v.p[k] = ptx::pair(t.x, t.y);
    }
}

template <typename T>
__device__ __forceinline__ void store_pairs(T* row, int c, int cols, const Eight& v) {
    uint16_t* at = reinterpret_cast<uint16_t*>(row) + pair_column(c, 0);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = ptx::unpair(v.p[k]);
        w[k] = pack2<T>(t.x, t.y);
    }
    if ((c | 255) < cols) {
        if ((reinterpret_cast<uintptr_t>(row) & 3u) == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(at + 64 * k) = w[k];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                at[64 * k] = static_cast<uint16_t>(w[k]);
                at[64 * k + 1] = static_cast<uint16_t>(w[k] >> 16);
            }
        }
    } else {
        const int left = cols - pair_column(c, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (left > 64 * k) at[64 * k] = static_cast<uint16_t>(w[k]);
            if (left > 64 * k + 1) at[64 * k + 1] = static_cast<uint16_t>(w[k] >> 16);
        }
    }
}

// Zeros for the columns past the row's end.
__device__ __forceinline__ void keep_pairs(Eight& v, int c, int cols) {
    if ((c | 255) < cols) return;
    const int left = cols - pair_column(c, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = ptx::unpair(v.p[k]);
        v.p[k] = ptx::pair(left > 64 * k ? t.x : 0.0f, left > 64 * k + 1 ? t.y : 0.0f);
    }
}

__device__ __forceinline__ void load_pairs_any(const void* p, int dtype, int c, int cols, Eight& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float t[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = pair_column(c, k) + i;
            t[i] = at >= cols            ? 0.0f
                   : dtype == TILES_BF16 ? to_float(static_cast<const __nv_bfloat16*>(p)[at])
                   : dtype == TILES_F16  ? to_float(static_cast<const __half*>(p)[at])
                                         : static_cast<const float*>(p)[at];
        }
        v.p[k] = ptx::pair(t[0], t[1]);
    }
}

// As emit: the 128 columns that share a scale are two pairs of every lane.
template <typename T, bool FP8>
__device__ __forceinline__ void emit_pairs(const LayerArgs& a, int64_t row, int c, int cols, const Eight& d,
                                           uint64_t rstd, uint64_t shift, const Eight& w, const Eight& b) {
    Eight y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y.p[i] = ptx::fma2(ptx::fma2(d.p[i], rstd, shift), w.p[i], b.p[i]);
    if constexpr (FP8) {
        keep_pairs(y, c, cols);
        uint8_t* const to = static_cast<uint8_t*>(a.y) + row * a.ldy;
        const bool even = (reinterpret_cast<uintptr_t>(to) & 1u) == 0 && (c | 255) < cols;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float2 t[2] = {ptx::unpair(y.p[2 * half]), ptx::unpair(y.p[2 * half + 1])};
            float m = max3_abs_nan(max3_abs_nan(t[0].x, t[0].y, t[1].x), t[1].y, 0.0f);
            m = block_amax(m);
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float s = max_nan(__fdiv_rn(m, kE4m3Max), kTinyScale), inv = __frcp_rn(s);
#pragma unroll
            for (int k = 2 * half; k < 2 * half + 2; ++k) {
                const float2 q = t[k & 1];
                const uint32_t bytes =
                    __nv_cvt_float2_to_fp8x2(make_float2(q.x * inv, q.y * inv), __NV_SATFINITE, __NV_E4M3);
                const int at = pair_column(c, k);
                if (even) {
                    *reinterpret_cast<uint16_t*>(to + at) = static_cast<uint16_t>(bytes);
                } else {
                    if (at < cols) to[at] = static_cast<uint8_t>(bytes);
                    if (at + 1 < cols) to[at + 1] = static_cast<uint8_t>(bytes >> 8);
                }
            }
            const int block = (c & ~255) / kBlock + half;
            if ((threadIdx.x & 31) == 0 && block * kBlock < cols)
                a.scales[row * a.scale_row + block * a.scale_block] = s;
        }
    } else {
        store_pairs<T>(static_cast<T*>(a.y) + row * a.ldy, c, cols, y);
    }
}

template <typename T, int N, int VPT>
struct OddRing {
    static constexpr int PIECES = static_cast<int>(sizeof(T)) / 2;

    char* at;                                  // the row's of the first stage
    int pitch, stage_bytes;                    // from one matrix to the next, from one stage to the next

    static constexpr size_t bytes(int threads, int per_block) {
        return static_cast<size_t>(kStages) * N * per_block * (threads * VPT * PIECES + 2) * 16;
    }
    __device__ __forceinline__ explicit OddRing(uint4* smem) {
        const int row = (static_cast<int>(blockDim.x) * VPT * PIECES + 2) * 16;
        at = reinterpret_cast<char*>(smem) + threadIdx.y * row;
        pitch = blockDim.y * row;
        stage_bytes = N * pitch;
    }
    // Start the copies of a row.
    __device__ __forceinline__ void copy(int stage, int n, const T* row, int cols, const Extent& e) const {
        const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u);
        const int pieces = (s + cols * static_cast<int>(sizeof(T)) + 15) / 16;
        const char* from = reinterpret_cast<const char*>(row) - s;
        char* to = at + stage * stage_bytes + n * pitch;
        // What lies outside the matrix, of its first and its last row's pieces, is not read.
        const int first = from < e.from, last = pieces - (from + pieces * 16 > e.to);
#pragma unroll
        for (int j = 0; j <= VPT * PIECES; ++j) {
            const int i = j * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
            if (i >= first && i < last) ptx::cp_async_16(to + i * 16, from + i * 16);
        }
        if (first || last < pieces) copy_ends(to, from, pieces, e);
    }
    static __device__ __noinline__ void copy_ends(char* to, const char* from, int pieces, const Extent& e) {
        const int i = threadIdx.x * static_cast<int>(sizeof(T));
        if (i >= 16) return;
        for (int piece : {0, pieces - 1}) {
            const char* f = from + piece * 16 + i;
            if (f >= e.from && f < e.to) *reinterpret_cast<T*>(to + piece * 16 + i) = *reinterpret_cast<const T*>(f);
        }
    }
    // Vector j of a row whose first byte is the s-th of its first piece.
    __device__ __forceinline__ void read(int stage, int n, int j, int s, int cols, uint32_t (&w)[4]) const {
        load_words(at + stage * stage_bytes + n * pitch + s,
                   (j * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8, cols, w);
    }
    __device__ __forceinline__ void read(int stage, int n, int j, int s, int cols, Eight& v) const {
        uint32_t w[4];
        read(stage, n, j, s, cols, w);
        widen_words<T>(w, v);
    }
};

// Rows of a matrix, one after the other, `by` rows apart: where the one lies that is
// copied next, and where the one that is read starts in its first piece.
template <typename T>
struct Walk {
    const T* ahead;
    int64_t by;
    int at;

    __device__ __forceinline__ Walk(const void* p, int64_t row, int64_t rows_apart, int64_t ld)
        : ahead(static_cast<const T*>(p) + row * ld), by(rows_apart * ld),
          at(static_cast<int>(reinterpret_cast<uintptr_t>(ahead) & 15u)) {}
    __device__ __forceinline__ int next() const { return (at + static_cast<int>(by * sizeof(T))) & 15; }
};

// A row's threads have all copied (and waited for) what they have.
__device__ __forceinline__ void meet() {
    if (blockDim.x > 32) ptx::named_barrier(1 + threadIdx.y, blockDim.x);
    else __syncwarp();
}

template <typename T, int VPT, bool FP8, bool RES>
__global__ void __launch_bounds__(kRows)
    layernorm_odd_ring_kernel(const LayerArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[8][2][16 * 4];
    float(*const mine)[16 * 4] = slots[blockDim.x > 32 ? threadIdx.y : 0];
    clear_slots(&slots[0][0][0], sizeof(slots) / 4);
    const int step = blockDim.x * 8, tid = threadIdx.x, cols = static_cast<int>(a.cols);
    const OddRing<T, RES ? 2 : 1, VPT> ring(ring_smem);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y, ahead = row;
    const Extent of_x = extent_of<T>(a.x, a.rows, a.ldx, cols), of_r = extent_of<T>(a.residual, a.rows, a.ldr, cols);
    Walk<T> x(a.x, row, stride, a.ldx), r(a.residual, row, stride, RES ? a.ldr : 0);
    T* h = a.h ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
    auto fetch = [&](int stage) {
        if (ahead < a.rows) {
            ring.copy(stage, 0, x.ahead, cols, of_x);
            if constexpr (RES) ring.copy(stage, 1, r.ahead, cols, of_r);
        }
        ptx::cp_async_commit();
        ahead += stride;
        x.ahead += x.by;
        if constexpr (RES) r.ahead += r.by;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);
    Eight w[VPT], b[VPT], v[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        load_pairs_any(a.weight, a.weight_dtype, j * step + tid * 8, cols, w[j]);
        b[j].fill(0.0f);
        if (a.bias) load_pairs_any(a.bias, a.weight_dtype, j * step + tid * 8, cols, b[j]);
    }
    const float inv_n = 1.0f / static_cast<float>(cols);
    auto take = [&](int stage) {
        Eight all;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            ring.read(stage, 0, j, x.at, cols, v[j]);
            if constexpr (RES) {
                Eight q;
                ring.read(stage, 1, j, r.at, cols, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j].p[i] = ptx::add2(v[j].p[i], q.p[i]);
            }
            if (h) store_pairs<T>(h, j * step + tid * 8, cols, v[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) all.p[i] = j ? ptx::add2(all.p[i], v[j].p[i]) : v[j].p[i];
        }
        x.at = x.next();
        if constexpr (RES) r.at = r.next();
        if (h) h += stride * a.ldh;
        return all.sum();
    };
    ptx::cp_async_wait_groups<kStages - 2>();                  // the first two rows
    meet();
    float s[4];
    s[0] = row < a.rows ? take(0) : 0.0f;
    row_sums<4, 1, 16, true>(s, mine[1]);
    __syncwarp();
    fetch(0);
    float total = s[0];
    int stage = 0, turn = 0;
    for (; row < a.rows; row += stride, turn ^= 1) {
        Eight d[VPT], d1, d2;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const uint64_t less = ptx::pair(-total * inv_n, -total * inv_n);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[j].p[i] = ptx::add2(v[j].p[i], less);
            keep_pairs(d[j], j * step + tid * 8, cols);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d1.p[i] = j ? ptx::add2(d1.p[i], d[j].p[i]) : d[j].p[i];
                d2.p[i] = j ? ptx::fma2(d[j].p[i], d[j].p[i], d2.p[i]) : ptx::mul2(d[j].p[i], d[j].p[i]);
            }
        }
        s[0] = d1.sum();
        s[1] = d2.sum();
        s[2] = 0.0f;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        if (row + stride < a.rows) s[2] = take(stage);
        ptx::cp_async_wait_groups<kStages - 2>();              // the row after the next, for all after the barrier
        row_sums<4, 3, 16, true>(s, mine[turn]);
        __syncwarp();
        fetch(stage);
        total = s[2];
        const float off = s[0] * inv_n, rstd = inverse_root(s[1] * inv_n, off, a.eps);
        const uint64_t rstd2 = ptx::pair(rstd, rstd), shift = ptx::pair(-off * rstd, -off * rstd);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            emit_pairs<T, FP8>(a, row, j * step + tid * 8, cols, d[j], rstd2, shift, w[j], b[j]);
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

// What a row's four sums (of d, d^2, g = dy w and g d) make of its gradients:
//   dx = g rstd - level - (d - off) back,   dweight += dy (d - off) rstd.
struct RowFactors {
    uint64_t off, rstd, level, back;           // -off, rstd, -level, -back in pairs

    __device__ __forceinline__ RowFactors(const float* s, float inv_n, float eps) {
        const float o = s[0] * inv_n, r = inverse_root(s[1] * inv_n, o, eps);
        const float l = s[2] * inv_n * r, k = (s[3] - o * s[2]) * inv_n * r * r * r;
        off = ptx::pair(-o, -o);
        rstd = ptx::pair(r, r);
        level = ptx::pair(-l, -l);
        back = ptx::pair(-k, -k);
    }
};

// The sums that a vector adds (columns past the row's end hold zeros in d and g).
__device__ __forceinline__ void grad_sums(const Eight& d, const Eight& g, const Eight& w, float (&s)[4]) {
    Eight q, e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q.p[i] = ptx::mul2(d.p[i], d.p[i]);
        e.p[i] = ptx::mul2(g.p[i], w.p[i]);
    }
    s[0] += d.sum();
    s[1] += q.sum();
    s[2] += e.sum();
#pragma unroll
    for (int i = 0; i < 4; ++i) q.p[i] = ptx::mul2(e.p[i], d.p[i]);
    s[3] += q.sum();
}

// The same, kept in pairs until a thread's last vector: its first one, and the
// others.
__device__ __forceinline__ void first_sums(const Eight& d, const Eight& g, const Eight& w, Eight (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[0].p[i] = d.p[i];
        s[1].p[i] = ptx::mul2(d.p[i], d.p[i]);
        s[2].p[i] = ptx::mul2(g.p[i], w.p[i]);
        s[3].p[i] = ptx::mul2(s[2].p[i], d.p[i]);
    }
}

__device__ __forceinline__ void grad_sums(const Eight& d, const Eight& g, const Eight& w, Eight (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t gw = ptx::mul2(g.p[i], w.p[i]);
        s[0].p[i] = ptx::add2(s[0].p[i], d.p[i]);
        s[1].p[i] = ptx::fma2(d.p[i], d.p[i], s[1].p[i]);
        s[2].p[i] = ptx::add2(s[2].p[i], gw);
        s[3].p[i] = ptx::fma2(gw, d.p[i], s[3].p[i]);
    }
}

// A vector's dx (in o), and its parts of the weight's and the bias's gradient.
__device__ __forceinline__ void grad_vector(const RowFactors& f, const Eight& d, const Eight& g,
                                            const Eight& w, Eight& o, Eight& dw, Eight& db) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t e = ptx::add2(d.p[i], f.off), gr = ptx::mul2(g.p[i], f.rstd);
        db.p[i] = ptx::add2(db.p[i], g.p[i]);
        dw.p[i] = ptx::fma2(gr, e, dw.p[i]);
        o.p[i] = ptx::fma2(e, f.back, ptx::fma2(gr, w.p[i], f.level));
    }
}

// Each block sweeps rows, gridDim.x * blockDim.y apart; a thread keeps the same
// columns throughout, so its parts of the weight's and the bias's gradient
// stay in registers until the block's one write to `partials` (rows short
// enough for one warp go eight to a block, whose parts are added first).
// blockIdx.y picks a span of columns when a row is longer than one block holds
// (a vector a thread): each span then reads the whole row for the sums and
// writes its own columns.  (With spans from 512 threads on 2000 x 8001 f16 rows took
// 118 us, 75 with 1024; 13233 x 4161 fp32 598 and 296.)
template <typename T, bool VEC, bool SPANS>
__global__ void __launch_bounds__(kMaxThreads)
    layernorm_grad_kernel(const LayerGradArgs a) {
    __shared__ float slots[32 + 128];
    extern __shared__ float side[];                // weights; in the end, with blockDim.y > 1, the other warps' parts
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int step = blockDim.x * 8;
    const int cols = static_cast<int>(a.cols);
    const int first = static_cast<int>(blockIdx.y) * step;
    const int c = first + threadIdx.x * 8;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    Eight dw, db;
    dw.fill(0.0f);
    db.fill(0.0f);
    auto load = [&](const T* p, int at, Eight& v) {
        float t[8];
        load8<T, VEC>(p, at, cols, t);
        v.from(t);
    };
    auto load_weight = [&](int at, Eight& v) {
        float t[8];
        load8_any<VEC>(a.weight, a.weight_dtype, at, cols, t);
        v.from(t);
    };
    // A thread's own weights wait in shared memory: they would not fit its registers, and
    // from L1, in their type and twice a row, 8192 x 4001 f16 rows took 153 us, not 126.
    const int threads = blockDim.x * blockDim.y;
    ulonglong2* const kept = reinterpret_cast<ulonglong2*>(side) + threadIdx.y * blockDim.x + threadIdx.x;
    {
        Eight w;
        load_weight(c, w);
        kept[0] = make_ulonglong2(w.p[0], w.p[1]);
        kept[threads] = make_ulonglong2(w.p[2], w.p[3]);
    }
    auto own_weight = [&](Eight& w) {
        const ulonglong2 lo = kept[0], hi = kept[threads];
        w.p[0] = lo.x;
        w.p[1] = lo.y;
        w.p[2] = hi.x;
        w.p[3] = hi.y;
    };
    auto centre = [&](int at, Eight& v, float mean) {
        const uint64_t less = ptx::pair(-mean, -mean);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = ptx::add2(v.p[i], less);
        keep<VEC>(v, at, cols);
    };
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * blockDim.y) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* h = static_cast<const T*>(a.h) + row * a.ldh;
        const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
        Eight g, d, w, past;
        load(dy, c, g);
        load(h, c, d);
        // dh with the others where it is one load, after the sums where it is eight.
        if (VEC && dh) load(dh, c, past);
        own_weight(w);
        float m[1] = {d.sum()}, s[4];
        if constexpr (SPANS) {
            for (int c0 = 0; c0 < cols; c0 += step) {
                if (c0 == first) continue;
                Eight q;
                load(h, c0 + threadIdx.x * 8, q);
                m[0] += q.sum();
            }
        }
        row_sums<1, 1, 32, false>(m, slots);
        const float mean = m[0] * inv_n;
        centre(c, d, mean);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = 0.0f;
        grad_sums(d, g, w, s);
        if constexpr (SPANS) {
            for (int c0 = 0; c0 < cols; c0 += step) {
                if (c0 == first) continue;
                const int at = c0 + threadIdx.x * 8;
                Eight p, q, u;
                load(dy, at, p);
                load(h, at, q);
                load_weight(at, u);
                centre(at, q, mean);
                grad_sums(q, p, u, s);
            }
        }
        row_sums<4, 4, 32, false>(s, slots + 32);
        const RowFactors f(s, inv_n, a.eps);
        own_weight(w);
        if (!VEC && dh) load(dh, c, past);
        Eight o;
        grad_vector(f, d, g, w, o, dw, db);
        if (dh)
#pragma unroll
            for (int i = 0; i < 4; ++i) o.p[i] = ptx::add2(o.p[i], past.p[i]);
        float t[8];
        o.to(t);
        store8<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx, c, cols, t);
    }
    float tw[8], tb[8];
    dw.to(tw);
    db.to(tb);
    if (blockDim.y > 1) {                          // then blockDim.x == 32: one warp a row
        __syncthreads();
        if (threadIdx.y > 0)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                side[(threadIdx.y - 1) * 512 + i * 32 + threadIdx.x] = tw[i];
                side[(threadIdx.y - 1) * 512 + 256 + i * 32 + threadIdx.x] = tb[i];
            }
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                tw[i] += side[y * 512 + i * 32 + threadIdx.x];
                tb[i] += side[y * 512 + 256 + i * 32 + threadIdx.x];
            }
    }
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    store8<float, VEC>(out, c, cols, tw);
    store8<float, VEC>(out + a.cols, c, cols, tb);
}

// The same with the rows' pieces 16-byte aligned and the whole row among
// blockDim.x threads (gridDim.y == 1): one block an SM, blockDim.y rows at a
// time (their threads meet at barriers of their own, and add their parts of the
// gradients in the end), the next two on their way in.  The sums of one row go
// together with the mean of the next, so that a row costs one barrier.
// 8192 x 4096 bf16 rows with dh 51.3 us, the reduction's launch included: 78% of
// the measured copy bandwidth.  The instructions bound it (a vector a thread and
// twice the threads: 77.6 us; single fp32 additions instead of pairs: 60.6).
template <typename T, int VPT>
__global__ void __launch_bounds__(kRows)
    layernorm_grad_ring_kernel(const LayerGradArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float slots[8][2][16 * 8];          // rows of several warps: at most 8
    float(*const mine)[16 * 8] = slots[blockDim.x > 32 ? threadIdx.y : 0];
    clear_slots(&slots[0][0][0], sizeof(slots) / 4);
    const int step = blockDim.x * 8, tid = threadIdx.x, cols = static_cast<int>(a.cols);
    Ring<T, 3, VPT> ring(ring_smem, step, cols);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y, ahead = row;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy + tid * 8;
    const T* h = static_cast<const T*>(a.h) + row * a.ldh + tid * 8;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh + tid * 8 : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
    auto fetch = [&](int stage) {
        if (ahead < a.rows) {
            ring.copy(stage, 0, dy, step);
            ring.copy(stage, 1, h, step);
            if (dh) ring.copy(stage, 2, dh, step);
        }
        ptx::cp_async_commit();
        ahead += stride;
        dy += stride * a.lddy;
        h += stride * a.ldh;
        if (dh) dh += stride * a.lddh;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    Eight dw[VPT], db[VPT], w[VPT];
    float mask[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float t[8];
        load8_any<true>(a.weight, a.weight_dtype, j * step + tid * 8, cols, t);
        w[j].from(t);
        dw[j].fill(0.0f);
        db[j].fill(0.0f);
        mask[j] = ring.in[j] ? -1.0f / static_cast<float>(cols) : 0.0f;
    }
    const float inv_n = 1.0f / static_cast<float>(cols);
    auto sum_of = [&](int stage) {
        Eight all, v;
        ring.read(stage, 1, 0, all);
#pragma unroll
        for (int j = 1; j < VPT; ++j) {
            ring.read(stage, 1, j, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) all.p[i] = ptx::add2(all.p[i], v.p[i]);
        }
        return all.sum();
    };
    ptx::cp_async_wait_groups<kStages - 2>();
    float s[8];
    s[0] = row < a.rows ? sum_of(0) : 0.0f;
    row_sums<8, 1, 16, true>(s, mine[1]);
    float total = s[0];
    int stage = 0, turn = 0;
    for (; row < a.rows; row += stride, turn ^= 1) {
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        Eight d[VPT], g[VPT];
        {
            Eight sums[4];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const uint64_t less = ptx::pair(total * mask[j], total * mask[j]);
                ring.read(stage, 1, j, d[j]);
                ring.read(stage, 0, j, g[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[j].p[i] = ptx::add2(d[j].p[i], less);
                if (j == 0) first_sums(d[j], g[j], w[j], sums);
                else grad_sums(d[j], g[j], w[j], sums);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = sums[j].sum();
        }
        const int next = stage + 1 == kStages ? 0 : stage + 1;
        ptx::cp_async_wait_groups<kStages - 2>();
        s[4] = row + stride < a.rows ? sum_of(next) : 0.0f;
        row_sums<8, 5, 16, true>(s, mine[turn]);
        total = s[4];
        const RowFactors f(s, inv_n, a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            Eight o;
            float t[8];
            grad_vector(f, d[j], g[j], w[j], o, dw[j], db[j]);
            if (a.dh) {
                Eight q;
                ring.read(stage, 2, j, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) o.p[i] = ptx::add2(o.p[i], q.p[i]);
            }
            o.to(t);
            store8<T, true>(dx, j * step + tid * 8, cols, t);
        }
        dx += stride * a.lddx;
        stage = next;
    }
    float tw[VPT][8], tb[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        dw[j].to(tw[j]);
        db[j].to(tb[j]);
    }
    if (blockDim.y > 1) {
        // The ring's memory takes the other rows' parts (it holds more).
        float* side = reinterpret_cast<float*>(ring_smem);
        const int pitch = blockDim.x, part = VPT * 16 * pitch;
        __syncthreads();
        if (threadIdx.y > 0)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float* at = side + (threadIdx.y - 1) * part + (j * 8 + i) * 2 * pitch + tid;
                    at[0] = tw[j][i];
                    at[pitch] = tb[j][i];
                }
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float* at = side + y * part + (j * 8 + i) * 2 * pitch + tid;
                    tw[j][i] += at[0];
                    tb[j][i] += at[pitch];
                }
    }
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = j * step + tid * 8;
        if (c < cols)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4*>(out + c + i) =
                    make_float4(tw[j][i], tw[j][i + 1], tw[j][i + 2], tw[j][i + 3]);
                *reinterpret_cast<float4*>(out + a.cols + c + i) =
                    make_float4(tb[j][i], tb[j][i + 1], tb[j][i + 2], tb[j][i + 3]);
            }
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

constexpr int kLayerVpt = 2;

// Rows at a time of a block with the ring, and blocks: one an SM.
struct RingGeometry { int threads, per_block, blocks; };

RingGeometry ring_geometry(int64_t rows, int64_t cols, int sms, int vpt) {
    RingGeometry g;
    g.threads = static_cast<int>((cols + 32 * 8 * vpt - 1) / (32 * 8 * vpt) * 32);
    g.per_block = std::max(1, kRows / g.threads);
    g.blocks = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>((rows + g.per_block - 1) / g.per_block, sms)));
    return g;
}

template <typename T, bool FP8, bool RES>
int launch_layer_ring(const LayerArgs& a, const RingGeometry& g, cudaStream_t st) {
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(layernorm_ring_kernel<T, kLayerVpt, FP8, RES>, kRingBytesMost, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    const size_t smem = std::max(Ring<T, RES ? 2 : 1, kLayerVpt>::BYTES, exact_smem(1));
    return launch(layernorm_ring_kernel<T, kLayerVpt, FP8, RES>, dim3(g.blocks),
                  dim3(g.threads, g.per_block), smem, st, a);
}

template <typename T, bool FP8, bool RES>
int launch_layer_odd_ring(const LayerArgs& a, const RingGeometry& g, cudaStream_t st) {
    using R = OddRing<T, RES ? 2 : 1, kLayerVpt>;
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(layernorm_odd_ring_kernel<T, kLayerVpt, FP8, RES>, kRingBytesMost, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    const size_t smem = std::max(R::bytes(g.threads, g.per_block), exact_smem(1));
    return launch(layernorm_odd_ring_kernel<T, kLayerVpt, FP8, RES>, dim3(g.blocks), dim3(g.threads, g.per_block),
                  smem, st, a);
}

template <typename T>
int launch_layer_any(const LayerArgs& a, bool vec, bool fp8, int sms, cudaStream_t st) {
    if constexpr (sizeof(T) == 2) {
        const RingGeometry g = ring_geometry(a.rows, a.cols, sms, kLayerVpt);
        // The ring pays where a row is more than a warp's vectors (16384 x 512
        // with residual 14.6 us against 18.9 without it, 16384 x 256 9.1
        // against 8.5), 16-bit (fp32: below), and where every row of a block
        // has a successor (2000 x 600: 5.8 against 4.8; 600 x 4096 6.9 against 7.8).
        const int64_t round = static_cast<int64_t>(g.per_block) * sms;
        const bool fits = a.cols > 256 && g.threads <= kRows;
        // Rows that start anywhere want some more rounds (2590 x 580 9.5 us, 7.6 without the
        // ring; 12000 x 301 13.0 against 15.1).
        if (!vec && fits && a.rows >= 4 * round) {
            if (a.residual)
                return fp8 ? launch_layer_odd_ring<T, true, true>(a, g, st)
                           : launch_layer_odd_ring<T, false, true>(a, g, st);
            return fp8 ? launch_layer_odd_ring<T, true, false>(a, g, st)
                       : launch_layer_odd_ring<T, false, false>(a, g, st);
        }
        if (vec && fits && a.rows >= 2 * round) {
            if (a.residual)
                return fp8 ? launch_layer_ring<T, true, true>(a, g, st)
                           : launch_layer_ring<T, false, true>(a, g, st);
            return fp8 ? launch_layer_ring<T, true, false>(a, g, st)
                       : launch_layer_ring<T, false, false>(a, g, st);
        }
    }
    if (vec) return fp8 ? launch_layer<T, true, true>(a, st) : launch_layer<T, true, false>(a, st);
    return fp8 ? launch_layer<T, false, true>(a, st) : launch_layer<T, false, false>(a, st);
}

// Vectors a thread in the ring: of fp32 one, whose two pieces fill as much of it.
constexpr int grad_vpt(int elem_bytes) { return elem_bytes == 2 ? 2 : 1; }

struct LayerGradGeometry { int threads, per_block, blocks, spans; };

// Without the ring: as many blocks as 1024 threads an SM allow, all spans' together.
LayerGradGeometry layer_grad_geometry(int64_t rows, int64_t cols, int sms) {
    LayerGradGeometry g;
    const int64_t vectors = (cols + 7) / 8;
    g.spans = static_cast<int>((vectors + kMaxThreads - 1) / kMaxThreads);
    g.threads = static_cast<int>(((vectors + g.spans - 1) / g.spans + 31) / 32 * 32);
    g.per_block = g.threads == 32 ? 8 : 1;
    const int64_t sweeps = (rows + g.per_block - 1) / g.per_block;
    const int per_sm = std::max(1, std::min(16, 1024 / (g.threads * g.per_block)));
    g.blocks = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(sweeps, static_cast<int64_t>(sms) * per_sm / g.spans)));
    return g;
}

// The 256-byte header and the partials of whichever form runs.
size_t layer_grad_bytes(int64_t rows, int64_t cols, int sms) {
    const int blocks = std::max(layer_grad_geometry(rows, cols, sms).blocks,
                                static_cast<int>(std::min<int64_t>(rows, sms)));
    return kConvMinWorkspaceBytes + static_cast<size_t>(std::max(1, blocks)) * static_cast<size_t>(cols) * 8;
}

int check_grad_sizes(int64_t rows, int64_t cols) {
    const int s = check_sizes(rows, cols);
    if (s == TILES_OK && cols > (1 << 28))            // (spans are a grid's second dimension)
        return fail(TILES_ERR_TOO_LARGE, "more than 2^28 columns");
    return s;
}

template <typename T>
int launch_layer_grad(const LayerGradArgs& a, bool vec, int sms, int* parts, cudaStream_t st) {
    constexpr int VPT = grad_vpt(sizeof(T));
    // fp32 rows fill the ring with half the threads' work: only while there are
    // few (300 x 4096: 14.3 us against 21.1 without it, 1500 x 4096 35.8 against
    // 37.5, 8192 x 4096 148 against 117).
    if (vec && a.cols <= kRows * 8 * VPT && (sizeof(T) == 2 || a.rows <= 10 * sms)) {
        const RingGeometry g = ring_geometry(a.rows, a.cols, sms, VPT);
        static std::atomic<uint64_t> opted{0};
        const cudaError_t e = opt_in_smem(layernorm_grad_ring_kernel<T, VPT>, kRingBytesMost, &opted);
        if (e != cudaSuccess) return static_cast<int>(e);
        *parts = g.blocks;
        return launch(layernorm_grad_ring_kernel<T, VPT>, dim3(*parts), dim3(g.threads, g.per_block),
                      std::max(Ring<T, 3, VPT>::BYTES, exact_smem(1)), st, a);
    }
    const LayerGradGeometry g = layer_grad_geometry(a.rows, a.cols, sms);
    *parts = g.blocks;
    const dim3 grid(g.blocks, g.spans), block(g.threads, g.per_block);
    const size_t side = std::max(g.threads * g.per_block * 32, (g.per_block - 1) * 512 * 4);
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
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    int e;
    if (d->dtype == TILES_BF16) e = launch_layer_any<__nv_bfloat16>(a, vec, fp8, sms, st);
    else if (d->dtype == TILES_F16) e = launch_layer_any<__half>(a, vec, fp8, sms, st);
    else e = launch_layer_any<float>(a, vec, fp8, sms, st);
    return launch_status(e, "layer norm");
}

size_t tiles_layernorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    if (check_grad_sizes(rows, cols) != TILES_OK) return 0;
    int sms = 0;
    if (current_sm_count(&sms) != TILES_OK) return 0;
    return layer_grad_bytes(rows, cols, sms);
}

int tiles_layernorm_grad(const tiles_layernorm_grad_desc* d, void* ws, size_t ws_bytes,
                         void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_grad_sizes(d->rows, d->cols);
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

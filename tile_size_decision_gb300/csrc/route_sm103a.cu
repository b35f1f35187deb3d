// Rows sorted by expert, and back: the stable sort of (token, choice) pairs by
// expert, the tokens' rows laid out in that order, the weighted sum that brings
// the experts' rows back, and its gradients.
//
// The sort is a counting sort of a few bytes a pair: launches and latency
// bound it.  The others move every row once: DRAM bounds them.
#include "row_ops.cuh"

namespace tiles {
namespace {

// ---- the sort -------------------------------------------------------------------

constexpr int kKeyBits = 13;                  // expert ids, and "none" (the number of groups)
constexpr int kMaxSortGroups = 4096;
constexpr int kMaxSortItems = 16;             // pairs a thread
constexpr int64_t kMaxSortPairs = 1 << 24;
static_assert(kMaxSortGroups < (1 << kKeyBits), "the id that stands for none fits");

struct SortArgs {
    const void* experts;
    int64_t ld;
    uint32_t pairs, k;
    int32_t groups;
    int32_t wide;                             // ids of 8 bytes
    int32_t* slots;
    int32_t* offsets;
    int32_t* order;
    uint16_t* counts;                         // [blocks][groups], with more than one block
};

// The expert of pair p, or `groups` where its id is none's.
__device__ __forceinline__ int expert_of(const SortArgs& a, uint32_t p) {
    const int64_t at = a.ld == a.k ? p : static_cast<int64_t>(p / a.k) * a.ld + p % a.k;
    if (a.wide) {
        const int64_t v = static_cast<const int64_t*>(a.experts)[at];
        return v >= 0 && v < a.groups ? static_cast<int>(v) : a.groups;
    }
    const int32_t v = static_cast<const int32_t*>(a.experts)[at];
    return v >= 0 && v < a.groups ? v : a.groups;
}

// Pairs of every expert in each block's share (I pairs a thread).
template <int I>
__global__ void __launch_bounds__(1024) sort_count_kernel(const SortArgs a) {
    extern __shared__ int count[];
    for (int g = threadIdx.x; g < a.groups; g += blockDim.x) count[g] = 0;
    __syncthreads();
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const uint32_t first = blockIdx.x * blockDim.x * I + threadIdx.x;
    int id[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t p = first + i * blockDim.x;
        id[i] = p < a.pairs ? expert_of(a, p) : a.groups;
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
        // One addition for all lanes of an expert: with a favourite expert 32
        // lanes would queue for one word.
        const uint32_t same = __match_any_sync(0xffffffffu, id[i]);
        if (id[i] < a.groups && (threadIdx.x & 31) == __ffs(same) - 1)
            atomicAdd(count + id[i], __popc(same));
    }
    __syncthreads();
    for (int g = threadIdx.x; g < a.groups; g += blockDim.x)
        a.counts[static_cast<int64_t>(blockIdx.x) * a.groups + g] = static_cast<uint16_t>(count[g]);
}

// The places of a block's pairs.  A warp takes 32 I consecutive pairs and ranks
// them among its own of the same expert; the warps' counts, those of the blocks
// before and the experts' totals then give every pair its row.  Everything
// is counted, nothing competes: the order is stable, and the same every time.
template <int I>
__global__ void __launch_bounds__(1024) sort_place_kernel(const SortArgs a) {
    extern __shared__ int start[];             // [groups]: totals, then the first row of the block's pairs
    __shared__ int sums[32];
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int warps = threads >> 5, groups = a.groups, pitch = (groups + 1) & ~1;
    int* below = start + groups;               // [groups]: pairs in the blocks before
    uint16_t* rank = reinterpret_cast<uint16_t*>(below + groups);   // [warps][pitch]
    for (int i = tid; i < warps * pitch / 2; i += threads) reinterpret_cast<uint32_t*>(rank)[i] = 0;
    for (int g = tid; g < groups; g += threads) start[g] = below[g] = 0;
    __syncthreads();
    // With several blocks the counting kernel went before.  It let this one start
    // after its own wait, so what came before it (the ids) is there: only the
    // counts have to be waited for, below.
    if (gridDim.x == 1) ptx::grid_dependency_wait();
    uint16_t* mine = rank + warp * pitch;
    const uint32_t first = blockIdx.x * threads * I + warp * 32 * I + lane;
    uint32_t key[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t p = first + i * 32;
        key[i] = p < a.pairs ? expert_of(a, p) : groups;
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int id = static_cast<int>(key[i]);
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const uint32_t before = id < groups ? mine[id] : 0;
        __syncwarp();
        if (id < groups && lane == __ffs(same) - 1) mine[id] = static_cast<uint16_t>(before + __popc(same));
        __syncwarp();
        key[i] |= (before + __popc(same & ((1u << lane) - 1))) << kKeyBits;
    }
    __syncthreads();
    // Counts of the warps to what lies before each of them.
    for (int g = tid; g < groups; g += threads) {
        int run = 0;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const int n = rank[w * pitch + g];
            rank[w * pitch + g] = static_cast<uint16_t>(run);
            run += n;
        }
        if (gridDim.x == 1) start[g] = run;
    }
    if (gridDim.x > 1) {
        ptx::grid_dependency_wait();
        // `side` threads share an expert's column of counts.
        const int side = max(1, threads / groups);
        for (int i = tid; i < side * groups; i += threads) {
            const int r = i / groups, g = i - r * groups;
            int all = 0, lower = 0;
#pragma unroll 8
            for (uint32_t b = r; b < gridDim.x; b += side) {
                const int n = a.counts[static_cast<int64_t>(b) * groups + g];
                all += n;
                lower += b < blockIdx.x ? n : 0;
            }
            atomicAdd(start + g, all);
            atomicAdd(below + g, lower);
        }
    }
    ptx::grid_launch_dependents();
    __syncthreads();
    // Totals to the experts' first rows.
    int placed = 0;
    for (int g0 = 0; g0 < groups; g0 += threads) {
        const int g = g0 + tid, n = g < groups ? start[g] : 0;
        int x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        const int s = lane < warps ? sums[lane] : 0;
        const int lower = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
        const int at = placed + lower + x - n;
        placed += __reduce_add_sync(0xffffffffu, s);
        if (g < groups) {
            if (blockIdx.x == 0) a.offsets[g] = at;
            start[g] = at + below[g];
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[groups] = placed;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t p = first + i * 32;
        if (p >= a.pairs) continue;
        const int id = static_cast<int>(key[i] & ((1u << kKeyBits) - 1));
        int row = -1;
        if (id < groups) {
            row = start[id] + mine[id] + static_cast<int>(key[i] >> kKeyBits);
            if (a.order) a.order[row] = static_cast<int32_t>(p);
        }
        a.slots[p] = row;
    }
    if (a.order)
        for (uint32_t p = placed + blockIdx.x * threads + tid; p < a.pairs; p += gridDim.x * threads)
            a.order[p] = -1;
}

struct SortGeometry { int threads, items, blocks; };

SortGeometry sort_geometry(int64_t pairs, int64_t groups) {
    SortGeometry g;
    // A warp's counts of 4096 experts are 8 KB.
    const int most = groups > 1024 ? 512 : 1024;
    g.threads = static_cast<int>(std::min<int64_t>(most, (std::max(pairs, groups) + 31) / 32 * 32));
    g.items = 1;
    // One block, one launch, for as long as a block has few pairs; then as many
    // blocks as there are SMs, of more pairs a thread where there are more.
    if (pairs <= 4 * static_cast<int64_t>(g.threads)) {
        while (pairs > static_cast<int64_t>(g.threads) * g.items) g.items *= 2;
    } else {
        while (g.items < kMaxSortItems && pairs > 152 * static_cast<int64_t>(g.threads) * g.items)
            g.items *= 2;
    }
    const int64_t share = static_cast<int64_t>(g.threads) * g.items;
    g.blocks = static_cast<int>(std::max<int64_t>(1, (pairs + share - 1) / share));
    return g;
}

size_t sort_bytes(int64_t pairs, int64_t groups) {
    const SortGeometry g = sort_geometry(pairs, groups);
    return kConvMinWorkspaceBytes +
           (g.blocks > 1 ? static_cast<size_t>(g.blocks) * static_cast<size_t>(groups) * 2 : 0);
}

template <int I>
int launch_sort(const SortArgs& a, const SortGeometry& g, cudaStream_t st) {
    const int pitch = (a.groups + 1) & ~1;
    const size_t smem = static_cast<size_t>(a.groups) * 8 + static_cast<size_t>(g.threads / 32) * pitch * 2;
    if (smem > 40 * 1024) {
        static std::atomic<uint64_t> opted{0};
        const cudaError_t e = opt_in_smem(sort_place_kernel<I>, kRingBytesMost, &opted);
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    if (g.blocks > 1) {
        const int e = launch(sort_count_kernel<I>, dim3(g.blocks), dim3(g.threads),
                             static_cast<size_t>(a.groups) * 4, st, a);
        if (e != cudaSuccess) return e;
    }
    return launch(sort_place_kernel<I>, dim3(g.blocks), dim3(g.threads), smem, st, a);
}

// ---- rows to the experts --------------------------------------------------------

struct DispatchArgs {
    int64_t tokens, rows, ld_slots;
    int32_t k;
    const int32_t* slots;
    const char* x;
    char* out;
    int64_t pitch_x, pitch_out;               // bytes
    int64_t pieces;                           // of sizeof(V) bytes, a row
    const float* scales;
    float* out_scales;
    int64_t scale_row, scale_block, out_scale_row, out_scale_block;
    int32_t blocks;                           // scales a row
    uint32_t row_grid;                        // blocks of the launch that move rows; the rest move scales
};

constexpr int kChoices = 8;                   // slots in registers at a time

// A token's row is read once and written to each of its slots.
template <typename V>
__global__ void __launch_bounds__(512) dispatch_kernel(const DispatchArgs a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (blockIdx.x >= a.row_grid) {
        // Scales: neighbours along whichever of rows and blocks lies together in
        // the output.
        const int64_t n = a.tokens * a.blocks;
        const int64_t step = static_cast<int64_t>(gridDim.x - a.row_grid) * blockDim.x * blockDim.y;
        for (int64_t i = (static_cast<int64_t>(blockIdx.x - a.row_grid) * blockDim.y + threadIdx.y) *
                             blockDim.x + threadIdx.x;
             i < n; i += step) {
            const bool along = a.out_scale_block == 1;
            const int64_t t = along ? i / a.blocks : i % a.tokens;
            const int64_t b = along ? i - t * a.blocks : i / a.tokens;
            const float s = a.scales[t * a.scale_row + b * a.scale_block];
            for (int j = 0; j < a.k; ++j) {
                const int32_t row = a.slots[t * a.ld_slots + j];
                if (row >= 0 && row < a.rows)
                    a.out_scales[row * a.out_scale_row + b * a.out_scale_block] = s;
            }
        }
        return;
    }
    const int64_t token = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (token >= a.tokens) return;
    const int32_t* slots = a.slots + token * a.ld_slots;
    const V* x = reinterpret_cast<const V*>(a.x + token * a.pitch_x);
    for (int j0 = 0; j0 < a.k; j0 += kChoices) {
        V* to[kChoices];
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
            const int32_t row = j0 + j < a.k ? slots[j0 + j] : -1;
            to[j] = row >= 0 && row < a.rows ? reinterpret_cast<V*>(a.out + row * a.pitch_out) : nullptr;
        }
        for (int64_t c = threadIdx.x; c < a.pieces; c += blockDim.x) {
            const V v = x[c];
#pragma unroll
            for (int j = 0; j < kChoices; ++j)
                if (to[j]) to[j][c] = v;
        }
    }
}

// ---- rows back to the tokens -----------------------------------------------------

struct CombineArgs {
    int64_t tokens, cols, rows, ld_slots;
    int32_t k;
    int32_t weight_dtype;
    const int32_t* slots;
    const void* weights;                      // or NULL: ones
    int64_t ld_weights;
    const void* in;                           // rows in expert order
    int64_t ld_in;
    const void* dy;                           // the gradient's: of y
    int64_t ld_dy;
    void* out;                                // y, or the rows' gradient
    int64_t ld_out;
    float* dweights;
    int64_t ld_dweights;
};

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
    if (dtype == TILES_F32) return static_cast<const float*>(p)[i];
    if (dtype == TILES_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

// Elements a thread moves at a time: 16 bytes, or one where rows start anywhere.
template <typename T, bool VEC>
struct Piece {
    static constexpr int N = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    uint4 q;
    T one;

    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC) q = *reinterpret_cast<const uint4*>(p);
        else one = *p;
    }
    __device__ __forceinline__ void clear() {
        if constexpr (VEC) q = make_uint4(0, 0, 0, 0);
        else one = from_float<T>(0.0f);
    }
    __device__ __forceinline__ void get(float (&v)[N]) const {
        if constexpr (!VEC) {
            v[0] = to_float(one);
        } else if constexpr (sizeof(T) == 4) {
            v[0] = __uint_as_float(q.x);
            v[1] = __uint_as_float(q.y);
            v[2] = __uint_as_float(q.z);
            v[3] = __uint_as_float(q.w);
        } else {
            const uint4 p[1] = {q};
            widen8<T>(p, v);
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[N]) {
        if constexpr (!VEC) {
            *p = from_float<T>(v[0]);
        } else if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                      pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
    }
};

// y[t] = the sum over the token's choices, in their order, in fp32.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) combine_kernel(const CombineArgs a) {
    using P = Piece<T, VEC>;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (token >= a.tokens) return;
    const int32_t* slots = a.slots + token * a.ld_slots;
    const T* in = static_cast<const T*>(a.in);
    T* y = static_cast<T*>(a.out) + token * a.ld_out;
    for (int64_t c = threadIdx.x * P::N; c < a.cols; c += blockDim.x * P::N) {
        float sum[P::N];
#pragma unroll
        for (int i = 0; i < P::N; ++i) sum[i] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kChoices) {
            P p[kChoices];
            float w[kChoices];
#pragma unroll
            for (int j = 0; j < kChoices; ++j) {
                const int32_t row = j0 + j < a.k ? slots[j0 + j] : -1;
                // A choice without an expert adds nothing, whatever its weight is.
                p[j].clear();
                w[j] = 0.0f;
                if (row >= 0 && row < a.rows) {
                    p[j].load(in + row * a.ld_in + c);
                    w[j] = a.weights ? load_any(a.weights, a.weight_dtype, token * a.ld_weights + j0 + j)
                                     : 1.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kChoices; ++j) {
                float v[P::N];
                p[j].get(v);
#pragma unroll
                for (int i = 0; i < P::N; ++i) sum[i] = fmaf(w[j], v[i], sum[i]);
            }
        }
        P::store(y + c, sum);
    }
}

// drows[slots[t][j]] = w[t][j] dy[t] and dw[t][j] = dy[t] . rows[slots[t][j]]: dy's
// row is read once for all choices, and every expert row as its gradient is
// written.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) combine_grad_kernel(const CombineArgs a) {
    using P = Piece<T, VEC>;
    __shared__ float part[kChoices][16];       // one warp a word, where a token has several
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = token < a.tokens;        // (all threads take part in the sums)
    const int32_t* slots = a.slots + token * a.ld_slots;
    const T* dy = static_cast<const T*>(a.dy) + token * a.ld_dy;
    const T* in = static_cast<const T*>(a.in);
    T* out = static_cast<T*>(a.out);
    for (int j0 = 0; j0 < a.k; j0 += kChoices) {
        int32_t row[kChoices];
        float w[kChoices], dot[kChoices];
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
            row[j] = live && j0 + j < a.k ? slots[j0 + j] : -1;
            if (row[j] >= a.rows) row[j] = -1;
            w[j] = row[j] >= 0 ? load_any(a.weights, a.weight_dtype, token * a.ld_weights + j0 + j) : 0.0f;
            dot[j] = 0.0f;
        }
        if (live)
            for (int64_t c = threadIdx.x * P::N; c < a.cols; c += blockDim.x * P::N) {
                P g, p[kChoices];
                g.load(dy + c);
#pragma unroll
                for (int j = 0; j < kChoices; ++j)
                    if (row[j] >= 0) p[j].load(in + row[j] * a.ld_in + c);
                float d[P::N];
                g.get(d);
#pragma unroll
                for (int j = 0; j < kChoices; ++j)
                    if (row[j] >= 0) {
                        float v[P::N], o[P::N];
                        p[j].get(v);
#pragma unroll
                        for (int i = 0; i < P::N; ++i) {
                            dot[j] = fmaf(d[i], v[i], dot[j]);
                            o[i] = d[i] * w[j];
                        }
                        P::store(out + row[j] * a.ld_out + c, o);
                    }
            }
        const int lanes = min(32, static_cast<int>(blockDim.x));
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
            for (int d = lanes >> 1; d >= 1; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
        if (blockDim.x > 32) {                 // then blockDim.y == 1
            const int warps = blockDim.x >> 5;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int j = 0; j < kChoices; ++j) part[j][threadIdx.x >> 5] = dot[j];
            __syncthreads();
            if (threadIdx.x < kChoices && j0 + static_cast<int>(threadIdx.x) < a.k) {
                float s = 0.0f;
                for (int i = 0; i < warps; ++i) s += part[threadIdx.x][i];
                a.dweights[token * a.ld_dweights + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        } else if (live && threadIdx.x == 0) {
#pragma unroll
            for (int j = 0; j < kChoices; ++j)
                if (j0 + j < a.k) a.dweights[token * a.ld_dweights + j0 + j] = dot[j];
        }
    }
}

// Threads a token and tokens a block: a power of two lanes for rows of a few
// pieces, else whole warps.
dim3 token_block(int64_t pieces) {
    if (pieces <= 32) {
        unsigned lanes = 1;
        while (lanes < pieces) lanes *= 2;
        return dim3(lanes, 256 / lanes);
    }
    const int64_t rounds = (pieces + 511) / 512;
    return dim3(static_cast<unsigned>(((pieces + rounds - 1) / rounds + 31) / 32 * 32), 1);
}

dim3 token_grid(int64_t tokens, dim3 block) {
    return dim3(static_cast<unsigned>((tokens + block.y - 1) / block.y));
}

template <typename V>
int launch_dispatch(DispatchArgs a, int sms, cudaStream_t st) {
    const dim3 block = token_block(a.pieces);
    dim3 grid = token_grid(a.tokens, block);
    a.row_grid = grid.x;
    if (a.scales) {
        const int64_t threads = static_cast<int64_t>(block.x) * block.y;
        grid.x += static_cast<unsigned>(
            std::min<int64_t>((a.tokens * a.blocks + threads - 1) / threads, 4 * static_cast<int64_t>(sms)));
    }
    return launch(dispatch_kernel<V>, grid, block, 0, st, a);
}

template <typename T>
int launch_combine(const CombineArgs& a, bool vec, bool grad, cudaStream_t st) {
    const int n = vec ? 16 / static_cast<int>(sizeof(T)) : 1;
    const dim3 block = token_block((a.cols + n - 1) / n), grid = token_grid(a.tokens, block);
    if (grad)
        return vec ? launch(combine_grad_kernel<T, true>, grid, block, 0, st, a)
                   : launch(combine_grad_kernel<T, false>, grid, block, 0, st, a);
    return vec ? launch(combine_kernel<T, true>, grid, block, 0, st, a)
               : launch(combine_kernel<T, false>, grid, block, 0, st, a);
}

// ---- checks ---------------------------------------------------------------------

int check_route(int64_t tokens, int64_t k, const int32_t* slots, int64_t ld_slots) {
    if (tokens < 0 || k < 1)
        return fail(TILES_ERR_INVALID_ARG, "tokens must be >= 0 and k >= 1 (tokens=%lld k=%lld)",
                    (long long)tokens, (long long)k);
    if (tokens > kMaxRows || k > kMaxRows || tokens * k > INT32_MAX)
        return fail(TILES_ERR_TOO_LARGE, "more than 2^31 - 1 pairs");
    if (tokens == 0) return TILES_OK;
    if (!slots || !element_aligned(slots, 4))
        return fail(TILES_ERR_INVALID_ARG, "slots is null or not aligned to its element");
    if (ld_slots < k) return fail(TILES_ERR_INVALID_ARG, "slots: row pitch smaller than the row length");
    return TILES_OK;
}

int check_combine(const tiles_combine_desc* d, bool grad) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_route(d->tokens, d->k, d->slots, d->ld_slots);
    if (s != TILES_OK) return s;
    if (d->rows < 0 || d->cols < 1)
        return fail(TILES_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (rows=%lld cols=%lld)",
                    (long long)d->rows, (long long)d->cols);
    if (d->rows > INT32_MAX || d->cols > kMaxRows) return fail(TILES_ERR_TOO_LARGE, "a size is too large");
    const int eb = dtype_bytes(d->dtype);
    if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the rows must be f16, bf16 or f32");
    if (d->tokens == 0) return TILES_OK;
    if (d->rows && (s = check_matrix("in", d->in, d->ld_in, d->cols, eb)) != TILES_OK) return s;
    if ((d->rows || !grad) && (s = check_matrix("out", d->out, d->ld_out, d->cols, eb)) != TILES_OK)
        return s;
    if (grad && !d->weights) return fail(TILES_ERR_INVALID_ARG, "weights is null");
    if (d->weights) {
        const int wb = dtype_bytes(d->weight_dtype);
        if (!wb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the weights must be f16, bf16 or f32");
        if (!element_aligned(d->weights, wb))
            return fail(TILES_ERR_MISALIGNED, "weights is not aligned to its element");
        if (d->ld_weights < d->k)
            return fail(TILES_ERR_INVALID_ARG, "weights: row pitch smaller than the row length");
    }
    if (grad) {
        if ((s = check_matrix("dy", d->dy, d->ld_dy, d->cols, eb)) != TILES_OK) return s;
        if (!d->dweights || !element_aligned(d->dweights, 4) || d->ld_dweights < d->k)
            return fail(TILES_ERR_INVALID_ARG,
                        "dweights is null, not aligned, or its row pitch smaller than the row length");
    }
    return TILES_OK;
}

int run_combine(const tiles_combine_desc* d, bool grad, void* stream) {
    const int s = check_combine(d, grad);
    if (s != TILES_OK || d->tokens == 0) return s;
    const int eb = dtype_bytes(d->dtype);
    const CombineArgs a{d->tokens, d->cols, d->rows, d->ld_slots, static_cast<int32_t>(d->k),
                        d->weight_dtype, d->slots, d->weights, d->ld_weights, d->in, d->ld_in, d->dy,
                        d->ld_dy, d->out, d->ld_out, d->dweights, d->ld_dweights};
    const bool vec = d->cols * eb % 16 == 0 && whole16(d->in, d->ld_in, eb) &&
                     whole16(d->out, d->ld_out, eb) && (!grad || whole16(d->dy, d->ld_dy, eb));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int e;
    if (d->dtype == TILES_BF16) e = launch_combine<__nv_bfloat16>(a, vec, grad, st);
    else if (d->dtype == TILES_F16) e = launch_combine<__half>(a, vec, grad, st);
    else e = launch_combine<float>(a, vec, grad, st);
    return launch_status(e, grad ? "combine gradient" : "combine");
}

}  // namespace
}  // namespace tiles

using namespace tiles;

extern "C" {

size_t tiles_expert_sort_workspace_bytes(int64_t tokens, int64_t k, int64_t groups) {
    if (tokens < 0 || k < 1 || groups < 1 || groups > kMaxSortGroups || tokens > kMaxSortPairs ||
        k > kMaxSortPairs || tokens * k > kMaxSortPairs) {
        fail(TILES_ERR_INVALID_ARG, "sizes out of range (tokens=%lld k=%lld groups=%lld)",
             (long long)tokens, (long long)k, (long long)groups);
        return 0;
    }
    return sort_bytes(tokens * k, groups);
}

int tiles_expert_sort(const tiles_expert_sort_desc* d, void* ws, size_t ws_bytes, void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    if (d->tokens < 0 || d->k < 1 || d->groups < 1)
        return fail(TILES_ERR_INVALID_ARG,
                    "tokens must be >= 0, k and groups >= 1 (tokens=%lld k=%lld groups=%lld)",
                    (long long)d->tokens, (long long)d->k, (long long)d->groups);
    if (d->groups > kMaxSortGroups)
        return fail(TILES_ERR_TOO_LARGE, "more than %d groups", kMaxSortGroups);
    if (d->tokens > kMaxSortPairs || d->k > kMaxSortPairs || d->tokens * d->k > kMaxSortPairs)
        return fail(TILES_ERR_TOO_LARGE, "more than 2^24 pairs");
    if (d->index_bytes != 4 && d->index_bytes != 8)
        return fail(TILES_ERR_UNSUPPORTED_DTYPE, "experts must be integers of 4 or 8 bytes");
    if (!d->offsets || !element_aligned(d->offsets, 4))
        return fail(TILES_ERR_INVALID_ARG, "offsets is null or not aligned to its element");
    const int64_t pairs = d->tokens * d->k;
    if (pairs) {
        if (!d->experts || !d->slots) return fail(TILES_ERR_INVALID_ARG, "experts or slots is null");
        if (!element_aligned(d->experts, d->index_bytes) || !element_aligned(d->slots, 4) ||
            !element_aligned(d->order, 4))
            return fail(TILES_ERR_MISALIGNED, "experts, slots or order is not aligned to its element");
        if (d->ld < d->k)
            return fail(TILES_ERR_INVALID_ARG, "experts: row pitch smaller than the row length");
    }
    const size_t need = sort_bytes(pairs, d->groups);
    if (!ws || ws_bytes < need)
        return fail(TILES_ERR_INVALID_ARG, "the sort needs %zu workspace bytes", need);
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(TILES_ERR_MISALIGNED, "the workspace must be 16-byte aligned");
    const SortArgs a{d->experts, d->tokens > 1 ? d->ld : d->k, static_cast<uint32_t>(pairs),
                     static_cast<uint32_t>(d->k), static_cast<int32_t>(d->groups),
                     d->index_bytes == 8, d->slots, d->offsets, d->order,
                     reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kConvMinWorkspaceBytes)};
    const SortGeometry g = sort_geometry(pairs, d->groups);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int e;
    switch (g.items) {
        case 1: e = launch_sort<1>(a, g, st); break;
        case 2: e = launch_sort<2>(a, g, st); break;
        case 4: e = launch_sort<4>(a, g, st); break;
        case 8: e = launch_sort<8>(a, g, st); break;
        default: e = launch_sort<16>(a, g, st); break;
    }
    return launch_status(e, "expert sort");
}

int tiles_expert_dispatch(const tiles_dispatch_desc* d, void* stream) {
    if (!d) return fail(TILES_ERR_INVALID_ARG, "null descriptor");
    int s = check_route(d->tokens, d->k, d->slots, d->ld_slots);
    if (s != TILES_OK) return s;
    if (d->rows < 0 || d->cols < 1)
        return fail(TILES_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (rows=%lld cols=%lld)",
                    (long long)d->rows, (long long)d->cols);
    if (d->rows > INT32_MAX || d->cols > kMaxRows) return fail(TILES_ERR_TOO_LARGE, "a size is too large");
    const int eb = d->dtype == TILES_E4M3 ? 1 : dtype_bytes(d->dtype);
    if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the rows must be f16, bf16, f32 or e4m3");
    if (d->tokens == 0 || d->rows == 0) return TILES_OK;
    if ((s = check_matrix("x", d->x, d->ldx, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("out", d->out, d->ld_out, d->cols, eb)) != TILES_OK) return s;
    if ((d->scales != nullptr) != (d->out_scales != nullptr))
        return fail(TILES_ERR_INVALID_ARG, "scales go with out_scales");
    if (!element_aligned(d->scales, 4) || !element_aligned(d->out_scales, 4))
        return fail(TILES_ERR_MISALIGNED, "the scales are not aligned to their element");
    const int64_t row_bytes = d->cols * eb;
    DispatchArgs a{d->tokens, d->rows, d->ld_slots, static_cast<int32_t>(d->k), d->slots,
                   static_cast<const char*>(d->x), static_cast<char*>(d->out), d->ldx * eb,
                   d->ld_out * eb, 0, d->scales, d->out_scales, d->scale_row, d->scale_block,
                   d->out_scale_row, d->out_scale_block,
                   static_cast<int32_t>((d->cols + kBlock - 1) / kBlock), 0};
    // The widest piece that every row is whole in.
    const uint64_t all = reinterpret_cast<uintptr_t>(d->x) | reinterpret_cast<uintptr_t>(d->out) |
                         static_cast<uint64_t>(row_bytes) |
                         static_cast<uint64_t>(d->tokens > 1 ? a.pitch_x : 0) |
                         static_cast<uint64_t>(d->rows > 1 ? a.pitch_out : 0);
    const int piece = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
    a.pieces = row_bytes / piece;
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int e;
    switch (piece) {
        case 16: e = launch_dispatch<uint4>(a, sms, st); break;
        case 8: e = launch_dispatch<uint2>(a, sms, st); break;
        case 4: e = launch_dispatch<uint32_t>(a, sms, st); break;
        case 2: e = launch_dispatch<uint16_t>(a, sms, st); break;
        default: e = launch_dispatch<uint8_t>(a, sms, st); break;
    }
    return launch_status(e, "dispatch");
}

int tiles_expert_combine(const tiles_combine_desc* d, void* stream) {
    return run_combine(d, false, stream);
}

int tiles_expert_combine_grad(const tiles_combine_desc* d, void* stream) {
    return run_combine(d, true, stream);
}

}  // extern "C"

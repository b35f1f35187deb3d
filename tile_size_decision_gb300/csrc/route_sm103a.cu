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
    int32_t* below;                           // [blocks][groups]: pairs in the blocks before; NULL: not
    int32_t* totals;                          // [groups], with below
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

// The blocks' counts of every expert to what lies before each block, and the
// totals: 32 experts a block, whose 32 rows of threads share the column.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const SortArgs a, int blocks) {
    __shared__ int sums[32][33];
    const int g = blockIdx.x * 32 + threadIdx.x, share = (blocks + 31) / 32;
    const int first = threadIdx.y * share, last = min(blocks, first + share);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const bool live = g < a.groups;
    int s = 0;
    if (live)
#pragma unroll 4
        for (int b = first; b < last; ++b) s += a.counts[static_cast<int64_t>(b) * a.groups + g];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    // Warp y adds up column y: lane i has the sum of the rows' shares up to i.
    int x = sums[threadIdx.x][threadIdx.y];
    const int n = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (static_cast<int>(threadIdx.x) >= d) x += y;
    }
    sums[threadIdx.x][threadIdx.y] = x - n;
    const int column = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 31 && column < a.groups) a.totals[column] = x;
    __syncthreads();
    if (!live) return;
    int run = sums[threadIdx.y][threadIdx.x];
    for (int b = first; b < last; ++b) {
        const int64_t at = static_cast<int64_t>(b) * a.groups + g;
        a.below[at] = run;
        run += a.counts[at];
    }
}

__host__ __device__ constexpr int rank_pitch(int groups) {
    // Counts of 16 bits: whole words, an odd number of them, so that the warps'
    // counts of one expert lie in different banks.
    return (groups + 1) / 2 % 2 ? (groups + 1) / 2 * 2 : (groups + 1) / 2 * 2 + 2;
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
    const int warps = threads >> 5, groups = a.groups, pitch = rank_pitch(groups);
    int* below = start + groups;               // [groups]: pairs in the blocks before
    uint16_t* rank = reinterpret_cast<uint16_t*>(below + groups);   // [warps][pitch]
    for (int i = tid; i < warps * pitch / 2; i += threads) reinterpret_cast<uint32_t*>(rank)[i] = 0;
    for (int g = tid; g < groups; g += threads) start[g] = below[g] = 0;
    __syncthreads();
    // The ids too are there only after this wait: that the counting kernel has waited for
    // them promises this one nothing.
    ptx::grid_dependency_wait();
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
    if (gridDim.x > 1 && a.below) {
        for (int g = tid; g < groups; g += threads) {
            start[g] = a.totals[g];
            below[g] = a.below[static_cast<int64_t>(blockIdx.x) * groups + g];
        }
    } else if (gridDim.x > 1) {
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

struct SortGeometry { int threads, items, blocks; bool scan; };

SortGeometry sort_geometry(int64_t pairs, int64_t groups) {
    SortGeometry g;
    g.items = 1;
    g.blocks = 1;
    g.scan = false;
    if (pairs <= 1024) {
        // One block, one launch (512 pairs among 64 experts 2.3 us; 4096 pairs 7.7, two
        // launches 4.8).  A warp's counts of 4096 experts are 8 KB.
        const int most = groups > 1024 ? 512 : 1024;
        g.threads = static_cast<int>(std::min<int64_t>(most, (std::max(pairs, groups) + 31) / 32 * 32));
        while (pairs > static_cast<int64_t>(g.threads) * g.items) g.items *= 2;
        return g;
    }
    // Blocks of 1024 pairs, of 512 where that leaves SMs without (131072 pairs
    // among 64 experts: 7.5 us, 10.4 with 1024 threads of a pair, 9.4 with 2048
    // pairs a block); more pairs a thread where there are more than two blocks
    // an SM.
    g.threads = pairs <= 65536 && groups <= 256 ? 256 : 512;
    g.items = 2;
    while (g.items < kMaxSortItems && pairs > 304 * static_cast<int64_t>(g.threads) * g.items) g.items *= 2;
    const int64_t share = static_cast<int64_t>(g.threads) * g.items;
    g.blocks = static_cast<int>((pairs + share - 1) / share);
    // Every block adds up the blocks' counts itself, or a launch of its own does:
    // 24 loads a thread are about a launch (131072 pairs: 64 experts 7.5 us against
    // 8.6, 256 experts 13.4 against 9.3, 4096 experts 106 against 18.4).
    g.scan = g.blocks > 1 && g.blocks * groups > 24 * static_cast<int64_t>(g.threads);
    return g;
}

// The header, the blocks' counts (whole 16 bytes), and what lies below each block
// with the totals.
size_t sort_counts_bytes(const SortGeometry& g, int64_t groups) {
    return (static_cast<size_t>(g.blocks) * static_cast<size_t>(groups) * 2 + 15) / 16 * 16;
}

size_t sort_bytes(int64_t pairs, int64_t groups) {
    const SortGeometry g = sort_geometry(pairs, groups);
    if (g.blocks == 1) return kConvMinWorkspaceBytes;
    return kConvMinWorkspaceBytes + sort_counts_bytes(g, groups) +
           (g.scan ? (static_cast<size_t>(g.blocks) + 1) * static_cast<size_t>(groups) * 4 : 0);
}

template <int I>
int launch_sort(const SortArgs& a, const SortGeometry& g, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(a.groups) * 8 +
                        static_cast<size_t>(g.threads / 32) * rank_pitch(a.groups) * 2;
    if (smem > 40 * 1024) {
        static std::atomic<uint64_t> opted{0};
        const cudaError_t e = opt_in_smem(sort_place_kernel<I>, kRingBytesMost, &opted);
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    int e = cudaSuccess;
    if (g.blocks > 1)
        e = launch(sort_count_kernel<I>, dim3(g.blocks), dim3(g.threads), static_cast<size_t>(a.groups) * 4, st, a);
    if (e == cudaSuccess && g.scan)
        e = launch(sort_scan_kernel, dim3((a.groups + 31) / 32), dim3(32, 32), 0, st, a, g.blocks);
    if (e != cudaSuccess) return e;
    return launch(sort_place_kernel<I>, dim3(g.blocks), dim3(g.threads), smem, st, a);
}

// ---- rows to the experts --------------------------------------------------------
//
// The kernels below that need no sum over a row see all tokens' rows as one run
// of pieces (16 bytes, or less where rows start anywhere): a thread takes the
// pieces u, u + stride, ..., whatever a row's length is, and no lane idles at a
// row's end.

// A thread's place in the run, advanced without a division.
struct Place {
    int64_t token;
    int32_t piece;

    __device__ __forceinline__ Place(int64_t u, int32_t pieces) {
        if (u >> 32) {
            token = u / pieces;
            piece = static_cast<int32_t>(u - token * pieces);
        } else {
            const uint32_t v = static_cast<uint32_t>(u), n = static_cast<uint32_t>(pieces);
            token = v / n;
            piece = static_cast<int32_t>(v - static_cast<uint32_t>(token) * n);
        }
    }
    __device__ __forceinline__ void advance(int64_t tokens, int32_t by, int32_t pieces) {
        token += tokens;
        piece += by;
        if (piece >= pieces) {
            piece -= pieces;
            ++token;
        }
    }
};

constexpr int kChoices = 8;                   // slots in registers at a time

// A token's slots j0 .. j0 + K - 1 as they are, -1 for those past the last.
// Nothing here looks at them: a loop that asks for the next token's while it
// works on one would wait for them at once.
template <int K>
__device__ __forceinline__ void load_slots(const int32_t* slots, int64_t ld, int64_t token, int j0, int k,
                                           bool live, int32_t (&row)[K]) {
    const int32_t* at = slots + token * ld + j0;
#pragma unroll
    for (int j = 0; j < K; ++j) row[j] = live && j0 + j < k ? at[j] : -1;
}

// Whether a slot is one of the rows.
__device__ __forceinline__ bool names(int32_t row, int64_t rows) {
    return static_cast<uint32_t>(row) < static_cast<uint32_t>(rows);   // rows are at most 2^31 - 1
}

// Rows that start anywhere: what is written is cut into pieces that start on 16
// bytes of its own row (the first and the last may be part of one); what is read
// for a piece is a window of the row.
// Piece c of a row of `bytes` (16 at least) that is written at `row`: the bytes
// [from, to) of the row, which may be none, and the 16 bytes of the row, from
// `window` on, that hold them.
struct Cut {
    int32_t from, to, window;

    __device__ __forceinline__ Cut(const void* row, int32_t bytes, int32_t c) {
        const int32_t first = c * 16 - static_cast<int32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
        from = max(first, 0);
        to = min(first + 16, bytes);
        window = min(from, bytes - 16);
    }
    __device__ __forceinline__ bool none() const { return from >= to; }
    __device__ __forceinline__ bool whole() const { return to - from == 16; }
    // Whether byte b of the window is one of the piece's.
    __device__ __forceinline__ bool has(int b) const { return window + b >= from && window + b < to; }
};

struct DispatchArgs {
    int64_t tokens, rows, ld_slots;
    int32_t k;
    int32_t pieces;                           // of sizeof(V) bytes, a row
    const int32_t* slots;
    const char* x;
    char* out;
    int64_t pitch_x, pitch_out;               // bytes
    const float* scales;
    float* out_scales;
    int64_t scale_row, scale_block, out_scale_row, out_scale_block;
    int32_t blocks;                           // scales a row
    uint32_t scale_grid;                      // blocks of the launch that move scales, before those for rows
    int32_t row_bytes, elem_bytes;
    int64_t near_tokens, step_tokens;         // what a thread advances by: to its next piece of
    int32_t near_pieces, step_pieces;         // the block's, and from past the last to the next round
};

constexpr int kMoveThreads = 256;

// Scales of 8-bit rows, by the first blocks of a launch (behind those that move
// rows they would end later: 8192 x 4 rows of 4096 e4m3 32.1 us against 28.2): neighbours
// along whichever of rows and blocks lies together in the output.
__device__ __forceinline__ void dispatch_scales(const DispatchArgs& a) {
    const int64_t n = a.tokens * a.blocks;
    const int64_t step = static_cast<int64_t>(a.scale_grid) * kMoveThreads;
    const bool along = a.out_scale_block == 1;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; i < n; i += step) {
        const int64_t t = along ? i / a.blocks : i % a.tokens;
        const int64_t b = along ? i - t * a.blocks : i / a.tokens;
        const float s = a.scales[t * a.scale_row + b * a.scale_block];
        for (int j = 0; j < a.k; ++j) {
            const int32_t row = a.slots[t * a.ld_slots + j];
            if (names(row, a.rows)) a.out_scales[row * a.out_scale_row + b * a.out_scale_block] = s;
        }
    }
}

// Rows that start and end on 16 bytes: a token's is read once and written to each
// of its slots; K: choices at a time, U: pieces of a thread in flight.
template <int K, int U>
__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const DispatchArgs a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (blockIdx.x < a.scale_grid) return dispatch_scales(a);
    const int64_t block = blockIdx.x - a.scale_grid;
    // A block takes U kMoveThreads pieces that lie together, then the same
    // gridDim.x times as far.
    Place at(block * (U * kMoveThreads) + threadIdx.x, a.pieces);
    while (at.token < a.tokens) {
        uint4 v[U];
        int32_t row[U][K], piece[U];
        int64_t token[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool live = at.token < a.tokens;
            token[u] = at.token;
            piece[u] = at.piece;
            load_slots<K>(a.slots, a.ld_slots, at.token, 0, a.k, live, row[u]);
            if (live) v[u] = reinterpret_cast<const uint4*>(a.x + at.token * a.pitch_x)[at.piece];
            at.advance(a.near_tokens, a.near_pieces, a.pieces);
        }
        at.advance(a.step_tokens, a.step_pieces, a.pieces);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (names(row[u][j], a.rows))
                    reinterpret_cast<uint4*>(a.out + row[u][j] * a.pitch_out)[piece[u]] = v[u];
            if (K == kChoices && token[u] < a.tokens)
                for (int j = K; j < a.k; ++j) {        // more than eight choices
                    const int32_t r = a.slots[token[u] * a.ld_slots + j];
                    if (names(r, a.rows)) reinterpret_cast<uint4*>(a.out + r * a.pitch_out)[piece[u]] = v[u];
                }
        }
    }
}

// The same for rows that start anywhere: a thread takes U pieces of one (token,
// choice) pair's row, a.pieces / U (rounded up) apart (a token's pairs are neighbours: x
// comes from L1 and L2).
template <int U>
__global__ void __launch_bounds__(kMoveThreads) dispatch_odd_kernel(const DispatchArgs a) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (blockIdx.x < a.scale_grid) return dispatch_scales(a);
    const int64_t block = blockIdx.x - a.scale_grid;
    const int32_t apart = (a.pieces + U - 1) / U;
    const Place at(block * kMoveThreads + threadIdx.x, apart);
    const int64_t pair = at.token, token = pair / a.k;
    if (token >= a.tokens) return;
    const int32_t row = a.slots[token * a.ld_slots + (pair - token * a.k)];
    if (!names(row, a.rows)) return;
    char* const out = a.out + row * a.pitch_out;
    const char* const x = a.x + token * a.pitch_x;
    if (a.row_bytes < 16) {                    // (then the row is one thread's)
        for (int b = at.piece == 0 ? 0 : 16; b < a.row_bytes; ++b) out[b] = x[b];
        return;
    }
    const Extent e{a.x, a.x + (a.tokens - 1) * a.pitch_x + a.row_bytes};
    Window w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Cut c(out, a.row_bytes, at.piece + u * apart);
        if (!c.none()) w[u].load(x + c.window, e, a.elem_bytes);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Cut c(out, a.row_bytes, at.piece + u * apart);
        if (c.none()) continue;
        const uint4 v = w[u].get();
        char* const to = out + c.window;
        if (c.whole()) {
            *reinterpret_cast<uint4*>(to) = v;
            continue;
        }
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
        if (a.elem_bytes == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c.has(4 * i)) reinterpret_cast<uint32_t*>(to)[i] = q[i];
        } else if (a.elem_bytes == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c.has(2 * i)) reinterpret_cast<uint16_t*>(to)[i] = static_cast<uint16_t>(q[i / 2] >> 16 * (i & 1));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c.has(i)) to[i] = static_cast<char>(q[i / 4] >> 8 * (i & 3));
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
    int64_t step_tokens;                      // what a thread advances by (the sum's)
    int32_t step_pieces, pieces;
};

// A token's weights j0 .. j0 + K - 1 (asked for beside its slots, not after them)
// as they lie in memory, and one of them as a number.
template <int K>
__device__ __forceinline__ void load_weights(const CombineArgs& a, int64_t token, int j0, bool live,
                                             uint32_t (&w)[K]) {
    const int64_t at = token * a.ld_weights + j0;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        w[j] = 0x3f800000u;                                    // 1
        if (a.weights && live && j0 + j < a.k)
            w[j] = a.weight_dtype == TILES_F32 ? static_cast<const uint32_t*>(a.weights)[at + j]
                                               : static_cast<const uint16_t*>(a.weights)[at + j];
    }
}

__device__ __forceinline__ float weight_of(const CombineArgs& a, uint32_t bits) {
    if (!a.weights || a.weight_dtype == TILES_F32) return __uint_as_float(bits);
    return a.weight_dtype == TILES_BF16 ? unpack2<__nv_bfloat16>(bits).x : unpack2<__half>(bits).x;
}

// 16 bytes of elements.
template <typename T>
struct Piece {
    static constexpr int N = 16 / static_cast<int>(sizeof(T));

    static __device__ __forceinline__ void widen(const uint4& q, float (&v)[N]) {
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
    static __device__ __forceinline__ void store(T* p, const float (&v)[N]) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                      pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
};

// y[t] = the sum over the token's choices, in their order, in fp32.  One piece a
// thread, its choices' loads in flight together.  K: choices at
// a time.  ODD: rows that start anywhere.
template <typename T, bool ODD, int K>
__global__ void __launch_bounds__(kMoveThreads) combine_kernel(const CombineArgs a) {
    using P = Piece<T>;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const Place at(static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x, a.pieces);
    if (at.token >= a.tokens) return;
    const T* in = static_cast<const T*>(a.in);
    T* y = static_cast<T*>(a.out) + at.token * a.ld_out;
    int64_t c = static_cast<int64_t>(at.piece) * P::N;
    constexpr int64_t kSize = sizeof(T);
    const bool small = ODD && a.cols * kSize < 16;             // (then the row is one thread's)
    const Cut cut(y, small ? 16 : static_cast<int32_t>(a.cols * kSize), at.piece);
    if constexpr (ODD) {
        if (small) {
            for (int64_t i = at.piece == 0 ? 0 : a.cols; i < a.cols; ++i) {
                float sum = 0.0f;
                for (int j = 0; j < a.k; ++j) {
                    const int32_t row = a.slots[at.token * a.ld_slots + j];
                    uint32_t w[1];
                    load_weights<1>(a, at.token, j, true, w);
                    if (names(row, a.rows)) sum = fmaf(weight_of(a, w[0]), to_float(in[row * a.ld_in + i]), sum);
                }
                y[i] = from_float<T>(sum);
            }
            return;
        }
        if (cut.none()) return;
        c = cut.window / kSize;
    }
    const Extent e = extent_of<T>(a.in, a.rows, a.ld_in, a.cols);
    // All choices' windows are asked for before the first is put together (1354 x 8 rows of
    // 314 bf16 columns 5.0 us against 8.6, 9328 x 3 of 205 7.5 against 8.8; 8000 x 4 of 1001
    // 30.2 against 28.2).
    in += c;
    float sum[P::N];
#pragma unroll
    for (int i = 0; i < P::N; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += K) {
        int32_t row[K];
        uint4 p[K];
        Window odd[ODD ? K : 1];
        uint32_t w[K];
        load_weights<K>(a, at.token, j0, true, w);
        load_slots<K>(a.slots, a.ld_slots, at.token, j0, a.k, true, row);
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (names(row[j], a.rows)) {
                const T* from = in + row[j] * a.ld_in;
                if constexpr (ODD) odd[j].load(reinterpret_cast<const char*>(from), e, sizeof(T));
                else p[j] = *reinterpret_cast<const uint4*>(from);
            }
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (names(row[j], a.rows)) {       // a choice without a row adds nothing, whatever its weight is
                const float f = weight_of(a, w[j]);
                float v[P::N];
                if constexpr (ODD) P::widen(odd[j].get(), v);
                else P::widen(p[j], v);
#pragma unroll
                for (int i = 0; i < P::N; ++i) sum[i] = fmaf(f, v[i], sum[i]);
            }
    }
    if (!ODD || cut.whole()) {
        P::store(y + c, sum);
    } else {
#pragma unroll
        for (int i = 0; i < P::N; ++i)
            if (cut.has(i * static_cast<int>(kSize))) y[c + i] = from_float<T>(sum[i]);
    }
}

// The same over many pieces, 16 bytes each: the next S - 1 pieces' rows on their
// way into shared memory while one is added up; what a thread copies only it
// reads, so that nothing waits for other threads.  K: choices, at most eight.
constexpr int kRingBlock = 512;

template <typename T, int K, int S>
__global__ void __launch_bounds__(kRingBlock) combine_ring_kernel(const CombineArgs a) {
    using P = Piece<T>;
    extern __shared__ uint4 ring_smem[];
    uint4* const ring = ring_smem + threadIdx.x;               // [S][K][threads]
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    Place ahead(static_cast<int64_t>(blockIdx.x) * kRingBlock + threadIdx.x, a.pieces), at = ahead;
    const T* in = static_cast<const T*>(a.in);
    auto look = [&](const Place& p, int32_t (&row)[K]) {
        load_slots<K>(a.slots, a.ld_slots, p.token, 0, a.k, p.token < a.tokens, row);
    };
    auto fetch = [&](int stage, const int32_t (&row)[K]) {      // the piece `ahead`
        const T* from = in + static_cast<int64_t>(ahead.piece) * P::N;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (names(row[j], a.rows))
                ptx::cp_async_16(ring + (stage * K + j) * kRingBlock, from + row[j] * a.ld_in);
        ptx::cp_async_commit();
        ahead.advance(a.step_tokens, a.step_pieces, a.pieces);
    };
    int32_t row[K], row_next[K];                               // of the piece added up now, and next
    uint32_t w[K], w_next[K];
    auto weigh = [&](const Place& p) {
        look(p, row_next);
        load_weights<K>(a, p.token, 0, p.token < a.tokens, w_next);
    };
    int32_t next[K];                                           // slots of `ahead`
    {
        int32_t first[S][K];
        Place p = ahead;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            look(p, first[i]);
            p.advance(a.step_tokens, a.step_pieces, a.pieces);
        }
        weigh(at);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) fetch(i, first[i]);
#pragma unroll
        for (int j = 0; j < K; ++j) next[j] = first[S - 1][j];
    }
    int stage = 0;
    while (at.token < a.tokens) {
        fetch(stage == 0 ? S - 1 : stage - 1, next);
        look(ahead, next);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            row[j] = row_next[j];
            w[j] = w_next[j];
        }
        T* const y = static_cast<T*>(a.out) + at.token * a.ld_out + static_cast<int64_t>(at.piece) * P::N;
        at.advance(a.step_tokens, a.step_pieces, a.pieces);
        weigh(at);
        ptx::cp_async_wait_groups<S - 1>();
        float sum[P::N];
#pragma unroll
        for (int i = 0; i < P::N; ++i) sum[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (names(row[j], a.rows)) {
                const float f = weight_of(a, w[j]);
                float v[P::N];
                P::widen(ring[(stage * K + j) * kRingBlock], v);
#pragma unroll
                for (int i = 0; i < P::N; ++i) sum[i] = fmaf(f, v[i], sum[i]);
            }
        P::store(y, sum);
        stage = stage + 1 == S ? 0 : stage + 1;
    }
}

// drows[slots[t][j]] = w[t][j] dy[t] and dw[t][j] = dy[t] . rows[slots[t][j]], one
// (token, choice) pair to blockDim.x threads: a power of two within a warp, or
// whole warps.  A token's pairs are neighbours, so that dy comes from DRAM once.
// ODD: rows that start anywhere, in pieces of drows' row.
template <typename T, bool ODD>
__global__ void __launch_bounds__(512) combine_grad_kernel(const CombineArgs a) {
    using P = Piece<T>;
    constexpr int kSize = sizeof(T);
    constexpr int U = 2;                       // pieces a thread has in flight
    __shared__ float part[16];                 // one warp a word, where a pair has several
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t token = pair / a.k;
    const int j = static_cast<int>(pair - token * a.k);
    const bool live = token < a.tokens;        // (all threads take part in the sum)
    int32_t row[1];
    uint32_t bits[1];
    load_weights<1>(a, token, j, live, bits);
    load_slots<1>(a.slots, a.ld_slots, token, j, a.k, live, row);
    float dot = 0.0f;
    if (names(row[0], a.rows)) {
        const T* dy = static_cast<const T*>(a.dy) + token * a.ld_dy;
        const T* from = static_cast<const T*>(a.in) + row[0] * a.ld_in;
        T* to = static_cast<T*>(a.out) + row[0] * a.ld_out;
        const float w = weight_of(a, bits[0]);
        const int32_t bytes = static_cast<int32_t>(a.cols * kSize);
        if (ODD && bytes < 16) {               // a row of less than a piece: its first thread's
            for (int i = threadIdx.x == 0 ? 0 : 16; i < a.cols; ++i) {
                const float d = to_float(dy[i]);
                dot = fmaf(d, to_float(from[i]), dot);
                to[i] = from_float<T>(d * w);
            }
        } else {
            const Extent of_dy = extent_of<T>(a.dy, a.tokens, a.ld_dy, a.cols);
            const Extent of_in = extent_of<T>(a.in, a.rows, a.ld_in, a.cols);
            for (int32_t p0 = threadIdx.x; p0 < a.pieces; p0 += U * static_cast<int32_t>(blockDim.x)) {
                uint4 g[U], q[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t piece = p0 + u * static_cast<int32_t>(blockDim.x);
                    if (piece >= a.pieces) continue;
                    if constexpr (ODD) {
                        const Cut cut(to, bytes, piece);
                        const char* d = reinterpret_cast<const char*>(dy) + cut.window;
                        const char* f = reinterpret_cast<const char*>(from) + cut.window;
                        if (cut.none()) continue;
                        g[u] = unaligned16(d, of_dy, kSize);
                        q[u] = unaligned16(f, of_in, kSize);
                    } else {
                        g[u] = reinterpret_cast<const uint4*>(dy)[piece];
                        q[u] = reinterpret_cast<const uint4*>(from)[piece];
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t piece = p0 + u * static_cast<int32_t>(blockDim.x);
                    const Cut cut(to, bytes, piece);
                    if (piece >= a.pieces || (ODD && cut.none())) continue;
                    float d[P::N], v[P::N], o[P::N];
                    P::widen(g[u], d);
                    P::widen(q[u], v);
#pragma unroll
                    for (int i = 0; i < P::N; ++i) {
                        const float f = fmaf(d[i], v[i], dot);
                        dot = !ODD || cut.has(i * kSize) ? f : dot;
                        o[i] = d[i] * w;
                    }
                    if (!ODD) {
                        P::store(to + static_cast<int64_t>(piece) * P::N, o);
                    } else if (cut.whole()) {
                        P::store(to + cut.window / kSize, o);
                    } else {
#pragma unroll
                        for (int i = 0; i < P::N; ++i)
                            if (cut.has(i * kSize)) to[cut.window / kSize + i] = from_float<T>(o[i]);
                    }
                }
            }
        }
    }
    const int lanes = min(32, static_cast<int>(blockDim.x));
    for (int d = lanes >> 1; d >= 1; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (blockDim.x > 32) {                     // then blockDim.y == 1
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i) dot += part[i];
    }
    if (live && threadIdx.x == 0) a.dweights[token * a.ld_dweights + j] = dot;
}

// The same over many tokens, in pieces of 16 bytes, V to a thread: blockDim.x
// threads a token (whole warps), blockDim.y tokens at a time, the next S - 1
// tokens' rows on their way into shared memory.  Each row of drows is written as
// its row is read, dy is read once for all K choices.
template <typename T, int K, int V, int S>
__global__ void __launch_bounds__(kRingBlock) combine_grad_ring_kernel(const CombineArgs a) {
    using P = Piece<T>;
    constexpr int STAGE = (K + 1) * V * kRingBlock;
    constexpr int KK = K <= 2 ? K : K <= 4 ? 4 : 8;            // the power of two from K on
    extern __shared__ uint4 ring_smem[];
    __shared__ float parts[8][2][16 * KK];                     // of tokens of several warps: [turn][warp][KK]
    uint4* const ring = ring_smem + threadIdx.y * blockDim.x + threadIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    const int c = tid * P::N, step = static_cast<int>(blockDim.x) * P::N;
    bool mine[V];
#pragma unroll
    for (int v = 0; v < V; ++v) mine[v] = v * static_cast<int>(blockDim.x) + tid < a.pieces;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t token = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y, ahead = token;
    const T* in = static_cast<const T*>(a.in) + c;
    T* out = static_cast<T*>(a.out) + c;
    auto look = [&](int64_t t, int32_t (&row)[K]) {
        load_slots<K>(a.slots, a.ld_slots, t, 0, a.k, t < a.tokens, row);
    };
    auto fetch = [&](int stage, const int32_t (&row)[K]) {      // the token `ahead`
        if (ahead < a.tokens) {
            const T* dy = static_cast<const T*>(a.dy) + ahead * a.ld_dy + c;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!mine[v]) continue;
                uint4* to = ring + stage * STAGE + v * kRingBlock;
                ptx::cp_async_16(to, dy + v * step);
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (names(row[j], a.rows))
                        ptx::cp_async_16(to + (j + 1) * V * kRingBlock, in + row[j] * a.ld_in + v * step);
            }
        }
        ptx::cp_async_commit();
        ahead += stride;
    };
    int32_t row[K], row_next[K];                               // of the token worked on now, and next
    uint32_t w[K], w_next[K];
    auto weigh = [&](int64_t t) {
        look(t, row_next);
        load_weights<K>(a, t, 0, t < a.tokens, w_next);
    };
    int32_t next[K];                                           // slots of `ahead`
    {
        int32_t first[S][K];
#pragma unroll
        for (int i = 0; i < S; ++i) look(ahead + i * stride, first[i]);
        weigh(token);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) fetch(i, first[i]);
#pragma unroll
        for (int j = 0; j < K; ++j) next[j] = first[S - 1][j];
    }
    int stage = 0, turn = 0;
    for (; token < a.tokens; token += stride, turn ^= 1) {
        fetch(stage == 0 ? S - 1 : stage - 1, next);
        look(ahead, next);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            row[j] = row_next[j];
            w[j] = w_next[j];
        }
        weigh(token + stride);
        ptx::cp_async_wait_groups<S - 1>();
        float dot[KK];
#pragma unroll
        for (int j = 0; j < KK; ++j) dot[j] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!mine[v]) continue;
            const uint4* from = ring + stage * STAGE + v * kRingBlock;
            float d[P::N];
            P::widen(from[0], d);
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (names(row[j], a.rows)) {
                    const float f = weight_of(a, w[j]);
                    float e[P::N], o[P::N];
                    P::widen(from[(j + 1) * V * kRingBlock], e);
#pragma unroll
                    for (int i = 0; i < P::N; ++i) {
                        dot[j] = fmaf(d[i], e[i], dot[j]);
                        o[i] = d[i] * f;
                    }
                    P::store(out + row[j] * a.ld_out + v * step, o);
                }
        }
        float x = fold<KK, K>(dot);            // lane l: the warp's sum of choice l % KK
        if (warps > 1) {
            float* at = parts[threadIdx.y][turn];
            if (lane < KK) at[(tid >> 5) * KK + lane] = x;
            ptx::named_barrier(1 + threadIdx.y, blockDim.x);
            if (tid < 32) {
                x = 0.0f;
                for (int i = lane; i < warps * KK; i += 32) x += at[i];
#pragma unroll
                for (int i = 16; i >= KK; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
            }
        }
        if (tid < a.k) a.dweights[token * a.ld_dweights + tid] = x;
        stage = stage + 1 == S ? 0 : stage + 1;
    }
}

// Threads a pair (two pieces or so each) and pairs a block: a power of two lanes
// for rows of a few pieces, else whole warps.
dim3 pair_block(int64_t pieces) {
    const int64_t want = (pieces + 1) / 2;
    if (want <= 32) {
        unsigned lanes = 1;
        while (lanes < want) lanes *= 2;
        return dim3(lanes, 256 / lanes);
    }
    const int64_t rounds = (want + 511) / 512;
    return dim3(static_cast<unsigned>(((want + rounds - 1) / rounds + 31) / 32 * 32), 1);
}

// Blocks that move scales.
unsigned scale_grid(const DispatchArgs& a, int sms) {
    if (!a.scales) return 0;
    return static_cast<unsigned>(std::min<int64_t>(
        (a.tokens * a.blocks + kMoveThreads - 1) / kMoveThreads, 2 * static_cast<int64_t>(sms)));
}

template <int K, int U>
int launch_dispatch(DispatchArgs a, int sms, cudaStream_t st) {
    // Every block one round (8192 x 4 rows of 4096 bf16 54 us, with 4 blocks an SM
    // that go round 63), as far as a grid goes.
    constexpr int64_t kShare = U * kMoveThreads;
    const int64_t grid = std::min<int64_t>((a.tokens * a.pieces + kShare - 1) / kShare, 1 << 30);
    a.near_tokens = kMoveThreads / a.pieces;
    a.near_pieces = kMoveThreads % a.pieces;
    a.step_tokens = (grid - 1) * kShare / a.pieces;
    a.step_pieces = static_cast<int32_t>((grid - 1) * kShare % a.pieces);
    a.scale_grid = scale_grid(a, sms);
    return launch(dispatch_kernel<K, U>, dim3(static_cast<unsigned>(grid) + a.scale_grid), dim3(kMoveThreads), 0,
                  st, a);
}

template <int U>
int launch_dispatch_odd(DispatchArgs a, int sms, cudaStream_t st) {
    const int64_t grid = (a.tokens * a.k * ((a.pieces + U - 1) / U) + kMoveThreads - 1) / kMoveThreads;
    if (grid > 1 << 30) return static_cast<int>(cudaErrorInvalidConfiguration);
    a.scale_grid = scale_grid(a, sms);
    return launch(dispatch_odd_kernel<U>, dim3(static_cast<unsigned>(grid) + a.scale_grid), dim3(kMoveThreads), 0, st,
                  a);
}

int launch_dispatch(DispatchArgs a, bool odd, int sms, cudaStream_t st) {
    if (odd) {
        a.pieces = static_cast<int32_t>((a.row_bytes + 14) / 16 + 1);
        // Four pieces a thread where there are threads enough and rows of some length (8000 x 4
        // rows of 1001 bf16 columns 22.8 us against 30.0 with one; 4 x 8 rows of 2001 2.7 against
        // 2.0, 8000 x 8 of 33 8.4 against 6.5).
        return a.pieces > 16 && a.tokens * a.k * a.pieces >= static_cast<int64_t>(sms) * 8 * kMoveThreads
                   ? launch_dispatch_odd<4>(a, sms, st) : launch_dispatch_odd<1>(a, sms, st);
    }
    a.pieces = static_cast<int32_t>(a.row_bytes / 16);
    if (a.k == 1) return launch_dispatch<1, 4>(a, sms, st);
    if (a.k <= 2) return launch_dispatch<2, 4>(a, sms, st);
    if (a.k <= 4) return launch_dispatch<4, 2>(a, sms, st);
    return launch_dispatch<kChoices, 2>(a, sms, st);
}

// PER: blocks an SM.
template <typename T, int K, int S, int PER>
int launch_combine_ring(CombineArgs a, int sms, cudaStream_t st) {
    constexpr size_t kBytes = static_cast<size_t>(S) * K * kRingBlock * 16;
    static_assert(kBytes <= kRingBytesMost && PER * (kBytes + 1024) <= 228 * 1024, "the blocks fit an SM");
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(combine_ring_kernel<T, K, S>, kRingBytesMost, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    const int64_t grid = std::min<int64_t>((a.tokens * a.pieces + kRingBlock - 1) / kRingBlock,
                                           static_cast<int64_t>(PER) * sms);
    a.step_tokens = grid * kRingBlock / a.pieces;
    a.step_pieces = static_cast<int32_t>(grid * kRingBlock % a.pieces);
    return launch(combine_ring_kernel<T, K, S>, dim3(static_cast<unsigned>(grid)), dim3(kRingBlock),
                  std::max(kBytes, exact_smem(PER)), st, a);
}

template <typename T, int K, int V, int S, int PER>
int launch_combine_grad_ring(const CombineArgs& a, int sms, cudaStream_t st) {
    constexpr size_t kBytes = static_cast<size_t>(S) * (K + 1) * V * kRingBlock * 16;
    static_assert(kBytes <= kRingBytesMost && PER * (kBytes + 1024) <= 228 * 1024, "the blocks fit an SM");
    static std::atomic<uint64_t> opted{0};
    const cudaError_t e = opt_in_smem(combine_grad_ring_kernel<T, K, V, S>, kRingBytesMost, &opted);
    if (e != cudaSuccess) return static_cast<int>(e);
    const unsigned threads = static_cast<unsigned>((a.pieces + 32 * V - 1) / (32 * V) * 32);
    const unsigned tokens = std::max(1u, kRingBlock / threads);
    const unsigned grid = static_cast<unsigned>(
        std::min<int64_t>((a.tokens + tokens - 1) / tokens, static_cast<int64_t>(PER) * sms));
    return launch(combine_grad_ring_kernel<T, K, V, S>, dim3(grid), dim3(threads, tokens), kBytes, st, a);
}

template <typename T>
int launch_combine_grad(CombineArgs a, bool odd, int sms, cudaStream_t st) {
    constexpr int64_t N = Piece<T>::N;
    a.pieces = static_cast<int32_t>(odd ? (a.cols * static_cast<int64_t>(sizeof(T)) + 14) / 16 + 1 : a.cols / N);
    // The ring takes tokens of some pieces where every block has a few of them
    // (500 x 4 rows of 2048 bf16: 6.4 us against 9.3 without it).  Two pieces a
    // thread make more of a token's fixed work (16000 rows of 4096 bf16, k 1: 64.8 us
    // against 75.3; 5333 x 3: 53.9 against 54.9) and take longer rows (4000 x 4 of
    // 8192: 101 us against 150 without the ring); one leaves room for more stages,
    // which k 4 is better off with (2048 columns: 51.2 us against 54.1) unless it
    // leaves threads idle (3000 columns: 44.6 against 38.4), and k 2 does
    // not care.  Beyond four choices two do not fit.
    if (!odd && a.k <= 8 && a.pieces > 16 && a.tokens >= 2 * sms) {
        const int threads = (a.pieces + 31) / 32 * 32;
        const bool idle = threads <= kRingBlock && kRingBlock / threads * threads < kRingBlock * 7 / 8;
        const bool two = a.pieces > kRingBlock || a.k == 1 || a.k == 3 || (a.k == 4 && idle);
        if (two && a.k <= 4 && a.pieces <= 2 * kRingBlock) {
            if (a.k == 1) return launch_combine_grad_ring<T, 1, 2, 3, 2>(a, sms, st);
            if (a.k == 2) return launch_combine_grad_ring<T, 2, 2, 4, 1>(a, sms, st);
            if (a.k == 3) return launch_combine_grad_ring<T, 3, 2, 3, 1>(a, sms, st);
            return launch_combine_grad_ring<T, 4, 2, 2, 1>(a, sms, st);
        }
        if (a.pieces <= kRingBlock) {
            if (a.k == 2) return launch_combine_grad_ring<T, 2, 1, 4, 2>(a, sms, st);
            if (a.k == 4) return launch_combine_grad_ring<T, 4, 1, 4, 1>(a, sms, st);
            if (a.k <= 6) return launch_combine_grad_ring<T, 6, 1, 3, 1>(a, sms, st);
            return launch_combine_grad_ring<T, 8, 1, 2, 1>(a, sms, st);
        }
    }
    const dim3 block = pair_block(a.pieces);
    const dim3 grid(static_cast<unsigned>((a.tokens * a.k + block.y - 1) / block.y));
    return odd ? launch(combine_grad_kernel<T, true>, grid, block, 0, st, a)
               : launch(combine_grad_kernel<T, false>, grid, block, 0, st, a);
}

template <typename T>
int launch_combine(CombineArgs a, bool odd, int sms, cudaStream_t st) {
    constexpr int64_t N = Piece<T>::N;
    a.pieces = static_cast<int32_t>(odd ? (a.cols * static_cast<int64_t>(sizeof(T)) + 14) / 16 + 1 : a.cols / N);
    const int64_t units = a.tokens * a.pieces;
    if (!odd && a.k <= 8 && units >= 4 * static_cast<int64_t>(sms) * kRingBlock) {
        // Threads an SM: as many as hold some 100 KB in flight (32768 rows of 2048
        // bf16: k 1 50 us with three blocks, 82 with one; k 2 35 against 50; k 4
        // 29.4 with two, 33.3 with one, 32.1 with three of fewer stages).
        if (a.k == 1) return launch_combine_ring<T, 1, 8, 3>(a, sms, st);
        if (a.k == 2) return launch_combine_ring<T, 2, 4, 3>(a, sms, st);
        if (a.k == 3) return launch_combine_ring<T, 3, 4, 2>(a, sms, st);
        if (a.k == 4) return launch_combine_ring<T, 4, 3, 2>(a, sms, st);
        if (a.k <= 6) return launch_combine_ring<T, 6, 2, 2>(a, sms, st);
        return launch_combine_ring<T, 8, 3, 1>(a, sms, st);
    }
    const int64_t grid = (units + kMoveThreads - 1) / kMoveThreads;
    if (grid > INT32_MAX) return static_cast<int>(cudaErrorInvalidConfiguration);
    const dim3 g(static_cast<unsigned>(grid)), b(kMoveThreads);
    if (a.k <= 4)
        return odd ? launch(combine_kernel<T, true, 4>, g, b, 0, st, a)
                   : launch(combine_kernel<T, false, 4>, g, b, 0, st, a);
    return odd ? launch(combine_kernel<T, true, 8>, g, b, 0, st, a)
               : launch(combine_kernel<T, false, 8>, g, b, 0, st, a);
}

// ---- checks ---------------------------------------------------------------------

constexpr int64_t kMaxCols = 1 << 28;          // the bytes of a row, and of its pieces, in 32 bits

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
    if (d->rows > INT32_MAX || d->cols > kMaxCols)
        return fail(TILES_ERR_TOO_LARGE, "more than 2^31 - 1 rows or 2^28 columns");
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
                        d->ld_dy, d->out, d->ld_out, d->dweights, d->ld_dweights, 0, 0, 0};
    // Whether every row starts and ends on 16 bytes.
    const uint64_t all = reinterpret_cast<uintptr_t>(d->in) | reinterpret_cast<uintptr_t>(d->out) |
                         static_cast<uint64_t>(d->cols * eb) |
                         static_cast<uint64_t>(d->rows > 1 ? d->ld_in * eb : 0) |
                         static_cast<uint64_t>((grad ? d->rows : d->tokens) > 1 ? d->ld_out * eb : 0) |
                         (grad ? reinterpret_cast<uintptr_t>(d->dy) |
                                     static_cast<uint64_t>(d->tokens > 1 ? d->ld_dy * eb : 0) : 0);
    const bool odd = all % 16 != 0;
    int sms = 0;
    const int q = current_sm_count(&sms);
    if (q != TILES_OK) return q;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto zero) {
        using T = decltype(zero);
        return grad ? launch_combine_grad<T>(a, odd, sms, st) : launch_combine<T>(a, odd, sms, st);
    };
    const int e = d->dtype == TILES_F32    ? go(float())
                  : d->dtype == TILES_BF16 ? go(__nv_bfloat16())
                                           : go(__half());
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
    if (need > kConvMinWorkspaceBytes && (!ws || ws_bytes < need))
        return fail(TILES_ERR_INVALID_ARG, "the sort needs %zu workspace bytes", need);
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(TILES_ERR_MISALIGNED, "the workspace must be 16-byte aligned");
    const SortGeometry g = sort_geometry(pairs, d->groups);
    char* const room = g.blocks > 1 ? static_cast<char*>(ws) + kConvMinWorkspaceBytes : nullptr;
    int32_t* const below = g.scan ? reinterpret_cast<int32_t*>(room + sort_counts_bytes(g, d->groups)) : nullptr;
    const SortArgs a{d->experts, d->tokens > 1 ? d->ld : d->k, static_cast<uint32_t>(pairs),
                     static_cast<uint32_t>(d->k), static_cast<int32_t>(d->groups),
                     d->index_bytes == 8, d->slots, d->offsets, d->order,
                     reinterpret_cast<uint16_t*>(room), below,
                     below ? below + static_cast<int64_t>(g.blocks) * d->groups : nullptr};
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
    if (d->rows > INT32_MAX || d->cols > kMaxCols)
        return fail(TILES_ERR_TOO_LARGE, "more than 2^31 - 1 rows or 2^28 columns");
    const int eb = d->dtype == TILES_E4M3 ? 1 : dtype_bytes(d->dtype);
    if (!eb) return fail(TILES_ERR_UNSUPPORTED_DTYPE, "the rows must be f16, bf16, f32 or e4m3");
    if (d->tokens == 0 || d->rows == 0) return TILES_OK;
    if ((s = check_matrix("x", d->x, d->ldx, d->cols, eb)) != TILES_OK) return s;
    if ((s = check_matrix("out", d->out, d->ld_out, d->cols, eb)) != TILES_OK) return s;
    if ((d->scales != nullptr) != (d->out_scales != nullptr))
        return fail(TILES_ERR_INVALID_ARG, "scales go with out_scales");
    if (!element_aligned(d->scales, 4) || !element_aligned(d->out_scales, 4))
        return fail(TILES_ERR_MISALIGNED, "the scales are not aligned to their element");
    DispatchArgs a{};
    a.tokens = d->tokens;
    a.rows = d->rows;
    a.ld_slots = d->ld_slots;
    a.k = static_cast<int32_t>(d->k);
    a.row_bytes = static_cast<int32_t>(d->cols * eb);
    a.elem_bytes = eb;
    a.slots = d->slots;
    a.x = static_cast<const char*>(d->x);
    a.out = static_cast<char*>(d->out);
    a.pitch_x = d->ldx * eb;
    a.pitch_out = d->ld_out * eb;
    a.scales = d->scales;
    a.out_scales = d->out_scales;
    a.scale_row = d->scale_row;
    a.scale_block = d->scale_block;
    a.out_scale_row = d->out_scale_row;
    a.out_scale_block = d->out_scale_block;
    a.blocks = static_cast<int32_t>((d->cols + kBlock - 1) / kBlock);
    // Whether every row starts and ends on 16 bytes.
    const uint64_t all = reinterpret_cast<uintptr_t>(d->x) | reinterpret_cast<uintptr_t>(d->out) |
                         static_cast<uint64_t>(a.row_bytes) |
                         static_cast<uint64_t>(d->tokens > 1 ? a.pitch_x : 0) |
                         static_cast<uint64_t>(d->rows > 1 ? a.pitch_out : 0);
    int sms = 0;
    if ((s = current_sm_count(&sms)) != TILES_OK) return s;
    const int e = launch_dispatch(a, all % 16 != 0, sms, static_cast<cudaStream_t>(stream));
    return launch_status(e, "dispatch");
}

int tiles_expert_combine(const tiles_combine_desc* d, void* stream) {
    return run_combine(d, false, stream);
}

int tiles_expert_combine_grad(const tiles_combine_desc* d, void* stream) {
    return run_combine(d, true, stream);
}

}  // extern "C"

// Host-side helpers of the kernels' launches, shared by the translation units
// of the norm and product operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "tiles_internal.h"

namespace tiles {

inline int dtype_bytes(int dtype) {
    return dtype == TILES_F16 || dtype == TILES_BF16 ? 2 : dtype == TILES_F32 ? 4 : 0;
}

// SM count of the current device (asked of the runtime once per device).
int current_sm_count(int* sms);

// TILES_OK, or TILES_ERR_CUDA with the runtime's text.
inline int launch_status(int e, const char* what) {
    if (e == cudaSuccess) return TILES_OK;
    return fail(TILES_ERR_CUDA, "%s launch failed: %s", what,
                cudaGetErrorString(static_cast<cudaError_t>(e)));
}

// Opts `kernel` into `bytes` of dynamic shared memory on the current device;
// remembered per device in the caller's `done` (one flag word per kernel), so
// that repeated launches ask the runtime nothing.
template <typename K>
cudaError_t opt_in_smem(K* kernel, int bytes, std::atomic<uint64_t>* done) {
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    const uint64_t bit = d < 64 ? uint64_t(1) << d : 0;
    if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// A launch with programmatic serialization (the kernel waits for its
// predecessor itself, before its first access to global memory) and, with
// cluster > 1, in clusters along x.  Returns a cudaError_t value.
template <typename... Params, typename... Args>
int launch_cluster(void (*kernel)(Params...), int cluster, dim3 grid, dim3 block, size_t smem,
                   cudaStream_t st, const Args&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return static_cast<int>(e);
    }
    return static_cast<int>(cudaSuccess);
}

template <typename... Params, typename... Args>
int launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
           const Args&... args) {
    return launch_cluster(kernel, 1, grid, block, smem, st, args...);
}

// A 3-D tensor map over a [d2][d1][d0] array of `type` elements (elem_bytes
// wide) with byte pitches, a box of {box0, box1, 1}, the 128-byte swizzle and
// zero fill out of range.
int encode_box(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t d0,
               uint64_t d1, uint64_t d2, uint64_t pitch1_bytes, uint64_t pitch2_bytes,
               uint32_t box0, uint32_t box1);

// The map through which whole 32-row x 64-byte boxes of an output leave (a
// [d2][d1][d0] array of F32, F16 or BF16, element pitches, 64-byte swizzle).
// False where TMA cannot address it (base or pitches not 16-byte multiples).
bool encode_out_boxes(CUtensorMap* map, int dtype, void* base, uint64_t d0, uint64_t d1,
                      uint64_t d2, uint64_t pitch1, uint64_t pitch2);

}  // namespace tiles

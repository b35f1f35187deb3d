// Host-side helpers declared in launch_util.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "launch_util.h"

namespace tiles {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cuTensorMapEncodeTiled through the runtime's driver entry point, so that
// the library loads without a GPU.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

}  // namespace

int encode_box(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t d0,
               uint64_t d1, uint64_t d2, uint64_t pitch1_bytes, uint64_t pitch2_bytes,
               uint32_t box0, uint32_t box1) {
    auto fn = encode_fn();
    if (!fn) return fail(TILES_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (no CUDA driver?)");
    cuuint64_t dims[3] = {d0, d1, d2};
    cuuint64_t strides[2] = {pitch1_bytes, pitch2_bytes};
    cuuint32_t box[3] = {box0, box1, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(TILES_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return TILES_OK;
}

bool encode_out_boxes(CUtensorMap* map, int dtype, void* base, uint64_t d0, uint64_t d1,
                      uint64_t d2, uint64_t pitch1, uint64_t pitch2) {
    auto fn = encode_fn();
    const uint64_t eb = dtype == TILES_F32 ? 4 : 2;
    if (!fn || !aligned16(base) || pitch1 * eb % 16 || pitch2 * eb % 16) return false;
    const CUtensorMapDataType t = dtype == TILES_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : dtype == TILES_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint64_t dims[3] = {d0, d1, d2};
    cuuint64_t strides[2] = {pitch1 * eb, pitch2 * eb};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(64 / eb), 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, t, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int current_sm_count(int* sms) {
    static std::atomic<int> known[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return fail(TILES_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    int n = d < 64 ? known[d].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
        if (e != cudaSuccess)
            return fail(TILES_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
        if (d < 64) known[d].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return TILES_OK;
}

}  // namespace tiles

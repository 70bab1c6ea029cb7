// delta_maps.cu -- tensor maps of the delta-rule kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "delta_chunk.cuh"

namespace ssd {
namespace delta {

cudaError_t encode_tiles(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                         const cuuint32_t *box) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    });
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box,
                          es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t same_tiles(CUtensorMap *m, const CUtensorMap &like, const void *base) {
    static PFN_cuTensorMapReplaceAddress_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapReplaceAddress_v12000)f;
    });
    if (!fn) return cudaErrorNotSupported;
    *m = like;
    return fn(m, const_cast<void *>(base)) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t allow_shared(const void *kernel, int bytes) {
    struct Seen {
        const void *kernel;
        int dev, bytes;
    };
    thread_local Seen seen[32];
    thread_local int count = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < count; ++i)
        if (seen[i].kernel == kernel && seen[i].dev == dev && seen[i].bytes == bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && count < 32) seen[count++] = Seen{kernel, dev, bytes};
    return e;
}

}  // namespace delta
}  // namespace ssd

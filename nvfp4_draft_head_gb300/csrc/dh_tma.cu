// Tensor maps (TMA descriptors), encoded by the driver on the host.
#include "dh_gemm.cuh"

namespace dh {
namespace gemm {

// The driver's encoder, looked up once (the library links against the runtime alone).
static cudaError_t encoder(PFN_cuTensorMapEncodeTiled_v12000* fn) {
    static std::atomic<void*> known{nullptr};
    void* p = known.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorNotSupported;
        known.store(p, std::memory_order_release);
    }
    *fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return cudaSuccess;
}

cudaError_t encode_map(CUtensorMap* map, const void* base, int elem, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    const cudaError_t e = encoder(&encode);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), box_rows}, one[2] = {1, 1};
    const auto call = [&] {
        return encode(map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides,
                      box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    if (r != CUDA_SUCCESS) {   // a thread that has made no runtime call yet has no context: bind the device's
        int dev = 0;
        cudaError_t bound = cudaGetDevice(&dev);
        if (bound == cudaSuccess) bound = cudaSetDevice(dev);
        if (bound != cudaSuccess) return bound;
        r = call();
    }
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace gemm
}  // namespace dh

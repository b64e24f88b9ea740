// sm100.cu -- host side of sm100.cuh: tensor maps, shared-memory limits.
#include "sm100.cuh"

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, through the runtime (the library does not link the driver); kept once it is found.
iqq_status encoder(EncodeTiled& fn)
{
    static std::atomic<EncodeTiled> known{nullptr};
    fn = known.load(std::memory_order_relaxed);
    if (fn != nullptr) return IQQ_OK;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess)
        return iqq::launch_status();
    if (found != cudaDriverEntryPointSuccess || p == nullptr) {
        iqq::set_last_cuda_error(cudaErrorNotSupported);
        return IQQ_ERR_CUDA;
    }
    fn = reinterpret_cast<EncodeTiled>(p);
    known.store(fn, std::memory_order_relaxed);
    return IQQ_OK;
}

}  // namespace

iqq_status iqq::byte_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t pitch, int box_rows)
{
    EncodeTiled fn;
    const iqq_status s = encoder(fn);
    if (s != IQQ_OK) return s;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t ones[2] = {1u, 1u};
    if (fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
        set_last_cuda_error(cudaErrorInvalidValue);
        return IQQ_ERR_CUDA;
    }
    return IQQ_OK;
}

iqq_status iqq::opt_in_smem(const void* kernel, size_t smem, std::atomic<uint64_t>& done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return launch_status();
    const uint64_t bit = dev < 64 ? 1ULL << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return IQQ_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return launch_status();
    done.fetch_or(bit, std::memory_order_relaxed);
    return IQQ_OK;
}

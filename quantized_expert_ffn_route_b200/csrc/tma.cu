// Host side of the tensor maps: the driver's encoder, looked up once.
#include "common.cuh"
#include "train/tma.cuh"

namespace moe {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

int make_tensor_map(CUtensorMap *map, const void *base, int bf16, uint64_t rows, uint64_t cols, uint64_t row_bytes,
                    uint32_t box_rows) {
    const EncodeTiled encode = encoder();
    if (!encode) {
        set_error("cuTensorMapEncodeTiled is not available in this driver");
        return MOE_ECUDA;
    }
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {row_bytes};
    const cuuint32_t box[2] = {64, box_rows}, steps[2] = {1, 1};
    const CUresult rc = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                               const_cast<void *>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (rc != CUDA_SUCCESS) {
        set_error("tensor map of %llu x %llu values refused (CUresult %d)", static_cast<unsigned long long>(rows),
                  static_cast<unsigned long long>(cols), static_cast<int>(rc));
        return MOE_ECUDA;
    }
    return MOE_OK;
}

int make_byte_map(CUtensorMap *map, const void *base, uint64_t rows, uint64_t bytes, uint32_t box_rows,
                  uint32_t box_bytes) {
    const EncodeTiled encode = encoder();
    if (!encode) {
        set_error("cuTensorMapEncodeTiled is not available in this driver");
        return MOE_ECUDA;
    }
    const cuuint64_t dims[2] = {bytes, rows}, strides[1] = {bytes};
    const cuuint32_t box[2] = {box_bytes, box_rows}, steps[2] = {1, 1};
    const CUresult rc = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, steps,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (rc != CUDA_SUCCESS) {
        set_error("tensor map of %llu x %llu bytes refused (CUresult %d)", static_cast<unsigned long long>(rows),
                  static_cast<unsigned long long>(bytes), static_cast<int>(rc));
        return MOE_ECUDA;
    }
    return MOE_OK;
}

}  // namespace moe

// Tensor maps of row-major matrices for 128-byte-swizzled K-major tiles (one
// 128-byte row in shared memory a matrix row), and the device's SM count.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lmoe {

enum class MapType {
    BF16,  // boxes of 64 columns
    FP4  // packed, two a byte in memory; 128 columns, a byte each in shared memory
};

// A map of [rows][K] elements (rows K elements apart) in boxes of box_rows rows.
inline bool make_tensor_map(CUtensorMap *m, const void *base, MapType type, int64_t K, int64_t rows, int box_rows)
{
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(type == MapType::BF16 ? 2 * K : K / 2)};
    const cuuint32_t box[2] = {type == MapType::BF16 ? 64u : 128u, cuuint32_t(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    const CUtensorMapDataType t =
        type == MapType::BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B;
    return encode(m, t, 2, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int device_sms()
{
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 152;
}

}  // namespace lmoe

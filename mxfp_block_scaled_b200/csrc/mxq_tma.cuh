// mxq_tma.cuh -- tensor maps of matrices, for cp.async.bulk.tensor (sm_100a).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxq {

// The driver's encoder of tensor maps (the library links the runtime only);
// its address, the same for every device, is looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled tensor_map_encoder()
{
    static const EncodeTiled encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return encode;
}

// Map of the row-major byte matrix [rows, cols] at p (16-byte aligned, cols a
// multiple of 16) in boxes of 128 bytes by box_rows (at most 256) rows, with
// the 128-byte swizzle: 16-byte piece i of row r of a box lies at piece
// i ^ (r % 8).  False where the encoder is missing or refuses.
inline bool make_byte_map(CUtensorMap *m, const uint8_t *p, uint64_t rows, uint64_t cols, uint32_t box_rows)
{
    const EncodeTiled encode = tensor_map_encoder();
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
    const cuuint32_t box[2] = {128, box_rows}, step[2] = {1, 1};
    return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(p), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of the row-major matrix [rows, cols] of bf16 or fp32 at p (16-byte
// aligned, rows of a multiple of 16 bytes) for stores of 128 bytes by box_rows
// rows from shared memory in the same swizzle.
inline bool make_out_map(CUtensorMap *m, void *p, uint64_t rows, uint64_t cols, bool f32, uint32_t box_rows)
{
    const EncodeTiled encode = tensor_map_encoder();
    const cuuint64_t size = f32 ? 4 : 2, dims[2] = {cols, rows}, strides[1] = {cols * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), box_rows}, step[2] = {1, 1};
    return encode && encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace mxq

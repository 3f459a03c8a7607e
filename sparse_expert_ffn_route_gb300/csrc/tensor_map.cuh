// tensor_map.cuh -- the driver's tensor map encoder (looked up once; null if there is none).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace moe {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// 2-D map of [rows][cols] elements, `ld` elements between rows, boxes of box_cols x box_rows
// with the 128-byte swizzle (box_cols elements are 128 bytes); what lies past the end reads as
// zero.  bits: 8 or 16 an element.
inline cudaError_t rows_map(CUtensorMap *m, const void *base, int bits, long long cols, long long ld, long long rows,
                            int box_rows)
{
    const auto enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * (bits / 8))};
    const cuuint32_t box[2] = {(cuuint32_t)(1024 / bits), (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, bits == 8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                           const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace moe

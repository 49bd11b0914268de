// Host helpers of the products: tensor maps and shared-memory limits.
// Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "csf_quant.cuh"

namespace csfk {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or null.
EncodeFn encode_fn();

// Raises a kernel's shared-memory limit once a device, to `limit` less what
// it has statically.  False on an error, and where the kernel was compiled to
// fewer than `least_regs` registers a thread.
bool allow_smem(const void *kernel, int limit, int least_regs = 0) noexcept;

// The map of a tensor of bytes; boxes of 128 bytes a row, 128-byte swizzle.
inline bool byte_map(CUtensorMap *map, const void *base, cuuint32_t rank, const cuuint64_t *dims, const cuuint64_t *strides,
                     const cuuint32_t *box) {
    const cuuint32_t ones[3] = {1, 1, 1};
    EncodeFn encode = encode_fn();
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void *>(base), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace csfk

// kda_tensor_map.h -- tensor maps of the tensor-core kernels (host side).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdint.h>

namespace kda {

// cuTensorMapEncodeTiled of the loaded driver, or nullptr (kda_prefill_tc.cu).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Map with 128-byte swizzled boxes (inner box extent 128 bytes), zeros outside
// the tensor.  Extents and strides from the inner dimension outwards; strides
// in bytes, without the inner one; base and strides multiples of 16.
inline bool make_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t d[5], s[5];
    cuuint32_t b[5], e[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i]; b[i] = box[i]; e[i] = 1;
        if (i + 1 < rank) s[i] = strides[i];
    }
    return enc(m, type, rank, const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda

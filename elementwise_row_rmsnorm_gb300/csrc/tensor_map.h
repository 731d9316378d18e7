// tensor_map.h -- descriptions of tensors for the tensor copies (TMA), made on
// the host.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace gbe {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        cudaGetLastError();
        return static_cast<EncodeFn>(nullptr);
    }();
    return fn;
}

inline bool encode(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* p, cuuint32_t rank,
                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return fn(m, type, rank, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 of `rank` dimensions, the innermost contiguous, the others `strides` bytes
// apart (of dimension 1 and on); copied in boxes, of the innermost 64 entries
// (128 bytes, swizzled by the place in shared memory); zeros outside.
inline bool encode_bf16(CUtensorMap* m, const void* p, cuuint32_t rank, const cuuint64_t* dims,
                        const cuuint64_t* strides, const cuuint32_t* box) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, p, rank, dims, strides, box);
}

// Bytes, row behind row.
inline bool encode_bytes(CUtensorMap* m, const void* p, cuuint32_t rank, const cuuint64_t* dims,
                         const cuuint64_t* strides, const cuuint32_t* box) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, p, rank, dims, strides, box);
}

}  // namespace gbe

// Tensor maps of the training kernels' TMA copies.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "train.h"

namespace mhc {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn()
{
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

bool encode_tensor(CUtensorMap *m, int esize, int rank, const void *base, const int64_t *dims,
            const int *box)
{
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[3], strides[2];
    cuuint32_t b[3], one[3] = {1, 1, 1};
    uint64_t stride = static_cast<uint64_t>(esize);
    for (int k = 0; k < rank; ++k) {
        d[k] = static_cast<cuuint64_t>(dims[k]);
        b[k] = static_cast<cuuint32_t>(box[k]);
        stride *= d[k];
        if (k + 1 < rank) strides[k] = stride;
    }
    const int row = box[0] * esize;
    const CUtensorMapSwizzle sw = row == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                  : row == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                              : CU_TENSOR_MAP_SWIZZLE_NONE;
    return fn(m, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, strides, b, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mhc

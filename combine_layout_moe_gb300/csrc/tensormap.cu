#include "tensormap.h"

namespace moe {

namespace {

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                            const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                            const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library links the runtime alone).
Encode encoder()
{
    static const Encode found = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    return found;
}

}  // namespace

namespace {

cudaError_t encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base,
                   const cuuint64_t *extents, const cuuint64_t *strides, const cuuint32_t *box)
{
    const Encode encode = encoder();
    if (encode == nullptr)
        return cudaErrorNotSupported;
    const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
    const CUresult st = encode(map, type, (cuuint32_t)rank, const_cast<void *>(base), extents,
                               strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return st == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t encode_map(CUtensorMap *map, CUtensorMapDataType type, int element, const void *base,
                       int64_t planes, int64_t rows, int64_t cols, int box_rows, int box_cols)
{
    const cuuint64_t extents[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)(cols * element),
                                   (cuuint64_t)(cols * element) * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    return encode(map, type, 3, base, extents, strides, box);
}

cudaError_t encode_map(CUtensorMap *map, CUtensorMapDataType type, const void *base,
                       const MapDim (&dims)[5])
{
    cuuint64_t extents[5], strides[4];
    cuuint32_t box[5];
    for (int i = 0; i < 5; i++) {
        extents[i] = (cuuint64_t)dims[i].extent;
        box[i] = (cuuint32_t)dims[i].box;
        if (i > 0)
            strides[i - 1] = (cuuint64_t)dims[i].stride;
    }
    return encode(map, type, 5, base, extents, strides, box);
}

}  // namespace moe

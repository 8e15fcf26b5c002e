// Host side of the tensor copies: encoding a tensor map.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

// A map of a dense row-major [planes, rows, cols] array in boxes of box_rows x
// box_cols (box_cols elements span at most 128 bytes), 128-byte swizzle, zeros
// outside.  Rows are cols * element size bytes, a multiple of 16.
cudaError_t encode_map(CUtensorMap *map, CUtensorMapDataType type, int element, const void *base,
                       int64_t planes, int64_t rows, int64_t cols, int box_rows, int box_cols);

// The same for any five dimensions (extent, stride in bytes, box), the first dense.
struct MapDim {
    int64_t extent, stride;
    int box;
};
cudaError_t encode_map(CUtensorMap *map, CUtensorMapDataType type, const void *base,
                       const MapDim (&dims)[5]);

}  // namespace moe

// The experts' row segments, as the products' kernels cut them into tiles, and
// the block quantisation that the products' epilogues share.
#pragma once

#include "common.cuh"

namespace moe {

// The rows of expert e, checked: an empty segment where the offsets descend or
// leave [0, N], which is reported.
__device__ __forceinline__ int2 segment(const int32_t *offsets, int e, int N, uint32_t *err_word)
{
    const int lo = offsets[e], hi = offsets[e + 1];
    if (lo < 0 || hi < lo || hi > N) {
        report(err_word, MOE_ERRBIT_BAD_INDEX);
        return make_int2(0, 0);
    }
    return make_int2(lo, hi);
}

struct Tile {
    int expert, row, rows;
};

// The `index`-th tile of `step` rows, the experts' segments one after another;
// rows == 0 behind the last.
__device__ inline Tile find_tile(const int32_t *offsets, int E, int N, int step, int index,
                                 uint32_t *err_word)
{
    Tile t = {0, 0, 0};
    for (int e = 0; e < E; e++) {
        const int2 s = segment(offsets, e, N, err_word);
        const int tiles = (s.y - s.x + step - 1) / step;
        if (index < tiles) {
            t.expert = e;
            t.row = s.x + index * step;
            t.rows = min(step, s.y - t.row);
            return t;
        }
        index -= tiles;
    }
    return t;
}

// Scale and reciprocal of a block whose largest magnitude is amax, each one
// correctly rounded division; a block of zeros, or one whose reciprocal
// overflows, has scale 1 and signed zero codes.
__device__ __forceinline__ void block_scale(float amax, float &scale, float &inv)
{
    scale = 1.0f;
    inv = 0.0f;
    if (amax > 0.0f) {
        const float r = __fdiv_rn(448.0f, amax);
        if (r <= 3.402823466e38f) {
            inv = r;
            scale = __fdiv_rn(amax, 448.0f);
        }
    }
}

}  // namespace moe

// Grouped FP8 products with block scales (sm_103a): moe_expert_gemm and
// moe_expert_swiglu.
//
// out[n, o] = sum_b sa[n, b] * S(e, o, b) * sum_{i in b} a[n, i] * W(e, o, i),
// with e the segment that holds row n and b the 128-wide blocks of the inputs.
//
// One CTA owns 32 rows of one expert and 128 outputs (for SwiGLU 128 gate
// and the matching 128 up outputs, so that a row's quantisation block is the
// CTA's own).  Codes widen to fp32 in shared memory, each block's products are
// summed and then scaled into the running fp32 sums.
#include <cuda_fp8.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "segments.cuh"

namespace moe {

namespace {

constexpr int GEMM_THREADS = 256;
constexpr int GEMM_ROWS = 32;
constexpr int GEMM_COLS = 128;
constexpr int GEMM_STEP = 32;

__device__ __forceinline__ float e4m3(uint8_t c)
{
    __nv_fp8_e4m3 v;
    v.__x = c;
    return static_cast<float>(v);
}

enum { OUT_ROWS_BF16, OUT_ROWS_F32, OUT_SWIGLU };

template <int OUT, bool TRANS>
__global__ void __launch_bounds__(GEMM_THREADS)
    expert_gemm_kernel(int N, int K, int M, int E, const uint8_t *__restrict__ a_q,
                       const float *__restrict__ a_s, const int32_t *__restrict__ offsets,
                       const uint8_t *__restrict__ w_q, const float *__restrict__ w_s,
                       void *__restrict__ out, float *__restrict__ out_s, uint32_t *err_word)
{
    constexpr int HALVES = OUT == OUT_SWIGLU ? 2 : 1;
    __shared__ float sa[GEMM_ROWS][GEMM_STEP + 1];
    __shared__ float sb[HALVES][GEMM_STEP][GEMM_COLS];
    __shared__ Tile tile;
    wait_prior_grid();
    if (threadIdx.x == 0)
        tile = find_tile(offsets, E, N, GEMM_ROWS, blockIdx.y, blockIdx.x == 0 ? err_word : nullptr);
    __syncthreads();
    if (tile.rows == 0)
        return;
    const int kb = K / 128, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int wide = OUT == OUT_SWIGLU ? 2 * M : M;
    const int ob = (wide + 127) / 128;
    const int o0 = blockIdx.x * GEMM_COLS;
    const int64_t wbase = (int64_t)tile.expert * wide * K;
    float acc[HALVES][4][4] = {}, part[HALVES][4][4];
    for (int b = 0; b < kb; b++) {
        for (int h = 0; h < HALVES; h++)
            for (int i = 0; i < 4; i++)
                for (int j = 0; j < 4; j++)
                    part[h][i][j] = 0.0f;
        for (int k0 = b * 128; k0 < (b + 1) * 128; k0 += GEMM_STEP) {
            __syncthreads();
            for (int i = threadIdx.x; i < GEMM_ROWS * GEMM_STEP; i += GEMM_THREADS) {
                const int r = i / GEMM_STEP, c = i % GEMM_STEP;
                sa[r][c] = r < tile.rows ? e4m3(a_q[(int64_t)(tile.row + r) * K + k0 + c]) : 0.0f;
            }
            for (int h = 0; h < HALVES; h++)
                for (int i = threadIdx.x; i < GEMM_COLS * GEMM_STEP; i += GEMM_THREADS) {
                    const int c = TRANS ? i % GEMM_COLS : i / GEMM_STEP;
                    const int r = TRANS ? i / GEMM_COLS : i % GEMM_STEP;
                    const int o = o0 + c;
                    const int64_t at = TRANS ? (int64_t)(k0 + r) * M + o
                                             : (int64_t)(o + h * M) * K + k0 + r;
                    sb[h][r][c] = o < M ? e4m3(w_q[wbase + at]) : 0.0f;
                }
            __syncthreads();
            for (int c = 0; c < GEMM_STEP; c++)
                for (int h = 0; h < HALVES; h++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            part[h][i][j] = fmaf(sa[ty * 4 + i][c], sb[h][c][tx + 32 * j],
                                                 part[h][i][j]);
        }
        for (int h = 0; h < HALVES; h++) {
            const int o = o0 / 128 + h * (M / 128);
            const float ws = w_s[(int64_t)tile.expert * ob * kb +
                                 (TRANS ? (int64_t)b * ob + o : (int64_t)o * kb + b)];
            for (int i = 0; i < 4; i++) {
                const int r = ty * 4 + i;
                const float s = r < tile.rows ? a_s[(int64_t)(tile.row + r) * kb + b] * ws : 0.0f;
                for (int j = 0; j < 4; j++)
                    acc[h][i][j] = fmaf(part[h][i][j], s, acc[h][i][j]);
            }
        }
    }
    for (int i = 0; i < 4; i++) {
        const int r = ty * 4 + i;
        if (r >= tile.rows)  // uniform in the warp
            continue;
        const int64_t n = tile.row + r;
        if constexpr (OUT == OUT_SWIGLU) {
            float h[4], amax = 0.0f;
            for (int j = 0; j < 4; j++) {
                const float g = acc[0][i][j];
                h[j] = g / (1.0f + expf(-g)) * acc[HALVES - 1][i][j];
                amax = fmaxf(amax, fabsf(h[j]));
            }
            for (int d = 16; d > 0; d >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, d));
            float scale = 1.0f, inv = 0.0f;
            block_scale(amax, scale, inv);
            for (int j = 0; j < 4; j++)
                static_cast<uint8_t *>(out)[n * M + o0 + tx + 32 * j] =
                    (uint8_t)__nv_cvt_float_to_fp8(__fmul_rn(h[j], inv), __NV_SATFINITE, __NV_E4M3);
            if (tx == 0)
                out_s[n * (M / 128) + o0 / 128] = scale;
        } else {
            for (int j = 0; j < 4; j++) {
                const int o = o0 + tx + 32 * j;
                if (o >= M)
                    continue;
                if constexpr (OUT == OUT_ROWS_F32)
                    static_cast<float *>(out)[n * M + o] = acc[0][i][j];
                else
                    static_cast<__nv_bfloat16 *>(out)[n * M + o] = __float2bfloat16_rn(acc[0][i][j]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_expert_gemm(int N, int K, int M, int E, const uint8_t *a_q, const float *a_s,
                               const int32_t *offsets, const uint8_t *w_q, const float *w_s,
                               bool transpose_w, void *out, bool out_f32, uint32_t *err_word,
                               cudaStream_t stream)
{
    if (N == 0)
        return cudaSuccess;
    const dim3 grid((M + GEMM_COLS - 1) / GEMM_COLS, (N + GEMM_ROWS - 1) / GEMM_ROWS + E);
    auto *kernel = transpose_w ? (out_f32 ? expert_gemm_kernel<OUT_ROWS_F32, true>
                                          : expert_gemm_kernel<OUT_ROWS_BF16, true>)
                               : (out_f32 ? expert_gemm_kernel<OUT_ROWS_F32, false>
                                          : expert_gemm_kernel<OUT_ROWS_BF16, false>);
    return launch_pdl(kernel, grid, dim3(GEMM_THREADS), 0, stream, N, K, M, E, a_q, a_s, offsets,
                      w_q, w_s, out, (float *)nullptr, err_word);
}

cudaError_t launch_expert_swiglu(int N, int K, int I, int E, const uint8_t *a_q, const float *a_s,
                                 const int32_t *offsets, const uint8_t *w_q, const float *w_s,
                                 uint8_t *h_q, float *h_s, uint32_t *err_word, cudaStream_t stream)
{
    if (N == 0)
        return cudaSuccess;
    const dim3 grid(I / GEMM_COLS, (N + GEMM_ROWS - 1) / GEMM_ROWS + E);
    return launch_pdl(expert_gemm_kernel<OUT_SWIGLU, false>, grid, dim3(GEMM_THREADS), 0, stream, N,
                      K, I, E, a_q, a_s, offsets, w_q, w_s, (void *)h_q, h_s, err_word);
}

}  // namespace moe

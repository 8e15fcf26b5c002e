// The experts' weight gradients (sm_103a): dw[e] = sum over e's rows of
// dy[n]^T x[n], bf16 in, fp32 out.
//
// One CTA owns a 64 x 64 tile of one expert's dw and walks the expert's rows
// sixteen at a time; products and sums are fp32.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "segments.cuh"

namespace moe {

namespace {

constexpr int WG_THREADS = 256;

__global__ void __launch_bounds__(WG_THREADS)
    expert_wgrad_kernel(int N, int M, int K, const __nv_bfloat16 *__restrict__ dy,
                        const __nv_bfloat16 *__restrict__ x, const int32_t *__restrict__ offsets,
                        float *__restrict__ dw, uint32_t *err_word)
{
    __shared__ float sy[16][64], sx[16][64];
    wait_prior_grid();
    const int e = blockIdx.z, m0 = blockIdx.y * 64, k0 = blockIdx.x * 64;
    const int2 s = segment(offsets, e, N, threadIdx.x == 0 ? err_word : nullptr);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int n0 = s.x; n0 < s.y; n0 += 16) {
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * 64; i += WG_THREADS) {
            const int r = i >> 6, c = i & 63;
            const bool in = n0 + r < s.y;
            sy[r][c] = in && m0 + c < M ? __bfloat162float(dy[(int64_t)(n0 + r) * M + m0 + c]) : 0;
            sx[r][c] = in && k0 + c < K ? __bfloat162float(x[(int64_t)(n0 + r) * K + k0 + c]) : 0;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 16; r++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    acc[i][j] = fmaf(sy[r][ty + 16 * i], sx[r][tx + 16 * j], acc[i][j]);
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++) {
            const int m = m0 + ty + 16 * i, c = k0 + tx + 16 * j;
            if (m < M && c < K)
                dw[((int64_t)e * M + m) * K + c] = acc[i][j];
        }
}

}  // namespace

cudaError_t launch_expert_wgrad(int N, int M, int K, int E, const void *dy, const void *x,
                                const int32_t *offsets, float *dw, uint32_t *err_word,
                                cudaStream_t stream)
{
    const dim3 grid((K + 63) / 64, (M + 63) / 64, E);
    return launch_pdl(expert_wgrad_kernel, grid, dim3(WG_THREADS), 0, stream, N, M, K,
                      static_cast<const __nv_bfloat16 *>(dy), static_cast<const __nv_bfloat16 *>(x),
                      offsets, dw, err_word);
}

}  // namespace moe

// A whole mixture-of-experts layer for a few tokens (sm_103a), in two kernels.
//
//   out[t] = sum_j w[t,j] * W2_e ( silu(Wg_e x[t]) * (Wu_e x[t]) ),  e = topk_idx[t,j]
//
// First kernel: a warp owns one (token, slot) pair and one inner channel: two
// dot products of length H, h = silu(g) * u in fp32 to the workspace.  Second: a
// warp owns one (token, output) and walks the token's slots.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int FEW_THREADS = 256;

__device__ __forceinline__ float weight(const uint8_t *w, int64_t at)
{
    __nv_fp8_e4m3 v;
    v.__x = w[at];
    return static_cast<float>(v);
}
__device__ __forceinline__ float weight(const __nv_bfloat16 *w, int64_t at)
{
    return __bfloat162float(w[at]);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

// This lane's part of row . x, with a scale for each 128 channels (or none).
template <typename W, typename X>
__device__ __forceinline__ float dot(const W *w, const float *scales, const X *x, int n, int lane)
{
    float sum = 0.0f;
    for (int c = lane; c < n; c += 32) {
        float v;
        if constexpr (sizeof(X) == 2)
            v = __bfloat162float(x[c]);
        else
            v = x[c];
        sum = fmaf(weight(w, c) * (scales ? scales[c >> 7] : 1.0f), v, sum);
    }
    return sum;
}

template <typename W>
__global__ void __launch_bounds__(FEW_THREADS)
    few_up_kernel(int T, int k, int H, int I, int E, const __nv_bfloat16 *__restrict__ x,
                  const int32_t *__restrict__ idx, const W *__restrict__ w13,
                  const float *__restrict__ s13, float *__restrict__ h, uint32_t *err_word)
{
    wait_prior_grid();
    allow_next_grid();
    const int lane = threadIdx.x & 31;
    const int pair = blockIdx.y, i = blockIdx.x * (FEW_THREADS / 32) + (threadIdx.x >> 5);
    const int e = idx[pair];
    if (e < 0 || e >= E) {
        if (threadIdx.x == 0 && blockIdx.x == 0)
            report(err_word, MOE_ERRBIT_BAD_INDEX);
        return;
    }
    if (i >= I)
        return;
    const int hb = H / 128;
    const int64_t g = (int64_t)e * 2 * I + i, u = g + I;
    const float *sg = s13 ? s13 + ((int64_t)e * (2 * I / 128) + i / 128) * hb : nullptr;
    const float *su = s13 ? sg + (int64_t)(I / 128) * hb : nullptr;
    const __nv_bfloat16 *row = x + (int64_t)(pair / k) * H;
    const float a = warp_sum(dot(w13 + g * H, sg, row, H, lane));
    const float b = warp_sum(dot(w13 + u * H, su, row, H, lane));
    if (lane == 0)
        h[(int64_t)pair * I + i] = a / (1.0f + expf(-a)) * b;
}

template <typename W>
__global__ void __launch_bounds__(FEW_THREADS)
    few_down_kernel(int T, int k, int H, int I, int E, const float *__restrict__ h,
                    const int32_t *__restrict__ idx, const float *__restrict__ topk_w,
                    const W *__restrict__ w2, const float *__restrict__ s2,
                    void *__restrict__ out, bool out_f32)
{
    wait_prior_grid();
    allow_next_grid();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.y, o = blockIdx.x * (FEW_THREADS / 32) + (threadIdx.x >> 5);
    if (o >= H)
        return;
    float sum = 0.0f;
    for (int j = 0; j < k; j++) {
        const int e = idx[t * k + j];
        if (e < 0 || e >= E)
            continue;
        const float *s = s2 ? s2 + ((int64_t)e * (H / 128) + o / 128) * (I / 128) : nullptr;
        const float y = dot(w2 + ((int64_t)e * H + o) * I, s, h + (int64_t)(t * k + j) * I, I, lane);
        sum = fmaf(topk_w[t * k + j], warp_sum(y), sum);
    }
    if (lane == 0) {
        const int64_t at = (int64_t)t * H + o;
        if (out_f32)
            static_cast<float *>(out)[at] = sum;
        else
            static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(sum);
    }
}

template <typename W>
cudaError_t layer(int T, int k, int H, int I, int E, const void *x, const int32_t *idx,
                  const float *topk_w, const void *w13, const float *s13, const void *w2,
                  const float *s2, void *out, bool out_f32, void *workspace, uint32_t *err_word,
                  cudaStream_t stream)
{
    constexpr int per = FEW_THREADS / 32;
    float *h = static_cast<float *>(workspace);
    cudaError_t st = launch_pdl(few_up_kernel<W>, dim3((I + per - 1) / per, T * k),
                                dim3(FEW_THREADS), 0, stream, T, k, H, I, E,
                                static_cast<const __nv_bfloat16 *>(x), idx,
                                static_cast<const W *>(w13), s13, h, err_word);
    if (st != cudaSuccess)
        return st;
    return launch_pdl(few_down_kernel<W>, dim3((H + per - 1) / per, T), dim3(FEW_THREADS), 0,
                      stream, T, k, H, I, E, (const float *)h, idx, topk_w,
                      static_cast<const W *>(w2), s2, out, out_f32);
}

}  // namespace

size_t layer_few_workspace_bytes(int T, int k, int H, int I)
{
    return (size_t)T * k * I * sizeof(float);
}

cudaError_t launch_layer_few(int T, int k, int H, int I, int E, const void *x, const int32_t *idx,
                             const float *topk_w, const void *w13, const float *s13,
                             const void *w2, const float *s2, bool fp8, void *out, bool out_f32,
                             void *workspace, uint32_t *err_word, cudaStream_t stream)
{
    if (T == 0)
        return cudaSuccess;
    return fp8 ? layer<uint8_t>(T, k, H, I, E, x, idx, topk_w, w13, s13, w2, s2, out, out_f32,
                                workspace, err_word, stream)
               : layer<__nv_bfloat16>(T, k, H, I, E, x, idx, topk_w, w13, nullptr, w2, nullptr,
                                      out, out_f32, workspace, err_word, stream);
}

}  // namespace moe

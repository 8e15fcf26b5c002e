// The experts' weight gradients (sm_103a): dw[e] = sum over e's rows n of
// dy[n]^T x[n], bf16 in, fp32 out.
//
// The sum runs over the rows, so both operands have their other index
// contiguous in memory (M of dy, K of x); the tensor core takes them as they lie.
// One persistent CTA per SM, 128 x 256 of one expert's dw a tile, 64 rows a stage:
//   warps 0-7   read a chunk's sums from tensor memory into their running sums
//               (thread: one o, 128 of the i), and store them after the last
//   warp 8      tensor copies of dy and x, 64 rows x 64 columns each
//   warp 9      issues the MMAs, K = 16 rows each; rows behind the segment's end
//               belong to the next expert and are zeroed in shared memory first
// The tensor core's fp32 sum truncates: 2.1e-6 relative after 2048 rows, growing
// with their number.  Each 1024 rows it starts from zero, and the chunks are added
// with rounding in registers.
#include "common.cuh"
#include "launch.h"
#include "segments.cuh"
#include "tcgen05.cuh"
#include "tensormap.h"

namespace moe {

namespace {

constexpr int W_THREADS = 384;  // three warpgroups
constexpr int W_SUMS = 256;     // threads of the first two
constexpr int W_M = 128;
constexpr int W_K = 256;
constexpr int W_STEP = 64;    // rows of a stage
constexpr int W_CHUNK = 1024; // rows the tensor core sums
constexpr int W_STAGES = 4;
constexpr int W_BOX = W_STEP * 128;  // bytes of 64 rows x 64 columns
constexpr int W_BOXES = (W_M + W_K) / 64;
constexpr int W_STAGE = W_BOXES * W_BOX;

struct WgradShared {
    uint64_t full[W_STAGES], empty[W_STAGES];
    uint64_t sums_full[2], sums_empty[2];
    uint32_t tmem;
    Segments seg;
};

constexpr size_t W_SMEM = 1024 + (size_t)W_STAGES * W_STAGE + sizeof(WgradShared);

struct WgradArgs {
    int N, M, K, E, m_tiles, k_tiles;
    const int32_t *offsets;
    float *dw;
    uint32_t *err_word;
};

struct WgradTile {
    int expert, lo, rows, m, k;
};

__device__ __forceinline__ WgradTile wgrad_tile(const Segments &s, const WgradArgs &g, int64_t tile)
{
    WgradTile t;
    const int per = g.m_tiles * g.k_tiles;
    t.expert = (int)(tile / per);
    const int local = (int)(tile - (int64_t)t.expert * per);
    t.m = local % g.m_tiles * W_M;
    t.k = local / g.m_tiles * W_K;
    t.lo = s.lo[t.expert];
    t.rows = s.hi[t.expert] - t.lo;
    return t;
}

__global__ void __launch_bounds__(W_THREADS, 1)
    expert_wgrad_kernel(const __grid_constant__ CUtensorMap map_dy,
                        const __grid_constant__ CUtensorMap map_x, const WgradArgs g)
{
    extern __shared__ uint8_t raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    WgradShared &sh = *reinterpret_cast<WgradShared *>(stages + W_STAGES * W_STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < W_STAGES; i++) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_addr(&sh.sums_full[i]), 1);
            mbar_init(smem_addr(&sh.sums_empty[i]), W_SUMS / 32);
        }
        mbar_fence_init();
        prefetch_map(&map_dy);
        prefetch_map(&map_x);
    }
    if (warp == 9)
        tmem_alloc(smem_addr(&sh.tmem), 512);
    wait_prior_grid();
    load_segments(sh.seg, g.offsets, g.E, g.N, [](int) { return 0; },
                  blockIdx.x == 0 ? g.err_word : nullptr);
    allow_next_grid();
    tcgen05_after_sync();
    const uint32_t tmem = sh.tmem;
    const int64_t tiles = (int64_t)g.E * g.m_tiles * g.k_tiles;
    bool ok = true;  // false once one of this warp's waits gave up

    // the sums' warps hold 128 running sums a thread: the third warpgroup gives
    // them its registers (168 at launch: 72 + 2 x 216 = 3 x 168)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            int s = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
                const WgradTile t = wgrad_tile(sh.seg, g, tile);
                for (int n = 0; n < t.rows; n += W_STEP) {
                    if (!(ok = warp_wait(smem_addr(&sh.empty[s]), phase ^ 1)))
                        break;
                    const uint32_t bar = smem_addr(&sh.full[s]);
                    const uint32_t at = smem_addr(stages + s * W_STAGE);
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar, W_STAGE);
#pragma unroll
                        for (int i = 0; i < W_M / 64; i++)
                            tensor_g2s(at + i * W_BOX, &map_dy, t.m + i * 64, t.lo + n, 0, bar);
#pragma unroll
                        for (int i = 0; i < W_K / 64; i++)
                            tensor_g2s(at + (W_M / 64 + i) * W_BOX, &map_x, t.k + i * 64, t.lo + n,
                                       0, bar);
                    }
                    issued++;
                    if (++s == W_STAGES) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            // copies still in flight land before the CTA may end
            for (int64_t i = issued > W_STAGES ? issued - W_STAGES : 0; i < issued; i++)
                ok = warp_wait(smem_addr(&sh.full[i % W_STAGES]), (i / W_STAGES) & 1) && ok;
        } else if (warp == 9) {
            constexpr uint32_t idesc = mma_desc(W_M, W_K, 1, true, true);
            const uint32_t base = smem_addr(stages);
            const uint64_t a0 = smem_desc(base, W_BOX, 1024);
            const uint64_t b0 = smem_desc(base + W_M / 64 * W_BOX, W_BOX, 1024);
            constexpr uint32_t k_step = 16 * 128 >> 4;  // sixteen rows on
            int s = 0, d = 0;
            uint32_t phase = 0, d_phase = 0;
            int64_t issued = 0;
            for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
                const WgradTile t = wgrad_tile(sh.seg, g, tile);
                for (int n = 0; n < t.rows; n += W_STEP) {
                    const bool first = n % W_CHUNK == 0;
                    const int left = t.rows - n;
                    const bool last = left <= W_STEP || (n + W_STEP) % W_CHUNK == 0;
                    if (!(ok = (!first || warp_wait(smem_addr(&sh.sums_empty[d]), d_phase ^ 1)) &&
                               warp_wait(smem_addr(&sh.full[s]), phase)))
                        break;
                    tcgen05_after_sync();
                    const int steps = left < W_STEP ? (left + 15) / 16 : W_STEP / 16;
                    if (left < steps * 16) {
                        const int pad = steps * 16 - left;  // rows of 128 bytes in each box
                        for (int i = lane; i < pad * W_BOXES * 8; i += 32) {
                            const int box = i / (pad * 8), in = i % (pad * 8);
                            *reinterpret_cast<uint4 *>(stages + s * W_STAGE + box * W_BOX +
                                                       left * 128 + in * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const uint64_t da = a0 + (uint32_t)(s * (W_STAGE >> 4));
                    const uint64_t db = b0 + (uint32_t)(s * (W_STAGE >> 4));
                    const uint32_t to = tmem + d * W_K;
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < W_STEP / 16; i++)
                            if (i < steps)
                                mma_bf16(to, da + i * k_step, db + i * k_step, idesc,
                                         !first || i > 0);
                        if (last)
                            tcgen05_commit(smem_addr(&sh.sums_full[d]));
                        tcgen05_commit(smem_addr(&sh.empty[s]));
                    }
                    issued++;
                    if (++s == W_STAGES) {
                        s = 0;
                        phase ^= 1;
                    }
                    if (last && ++d == 2) {
                        d = 0;
                        d_phase ^= 1;
                    }
                }
            }
            // and so do the MMAs' arrivals
            for (int64_t i = issued > W_STAGES ? issued - W_STAGES : 0; i < issued; i++)
                ok = warp_wait(smem_addr(&sh.empty[i % W_STAGES]), (i / W_STAGES) & 1) && ok;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp >> 2, quarter = warp & 3;
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
        int d = 0;
        uint32_t d_phase = 0;
        for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
            const WgradTile t = wgrad_tile(sh.seg, g, tile);
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; i++)
                acc[i] = 0.0f;
            for (int n = 0; n < t.rows; n += W_CHUNK) {
                if (!(ok = warp_wait(smem_addr(&sh.sums_full[d]), d_phase)))
                    break;
                tcgen05_after_sync();
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    uint32_t p[32];
                    tmem_ld32(mine + d * W_K + q * 32, p);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        acc[q * 32 + i] += __uint_as_float(p[i]);
                }
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.sums_empty[d]));
                if (++d == 2) {
                    d = 0;
                    d_phase ^= 1;
                }
            }
            if (!ok)
                break;
            const int m = t.m + quarter * 32 + lane, k = t.k + half * 128;
            if (m < g.M) {
                float *to = g.dw + ((int64_t)t.expert * g.M + m) * g.K + k;
#pragma unroll
                for (int v = 0; v < 32; v++)
                    if (k + v * 4 < g.K)
                        st_v4(to + v * 4, make_uint4(__float_as_uint(acc[4 * v]),
                                                     __float_as_uint(acc[4 * v + 1]),
                                                     __float_as_uint(acc[4 * v + 2]),
                                                     __float_as_uint(acc[4 * v + 3])));
            }
        }
    }
    if (!ok)
        report(g.err_word, MOE_ERRBIT_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    if (warp == 9)
        tmem_free(tmem, 512);
}

}  // namespace

cudaError_t launch_expert_wgrad(int N, int M, int K, int E, const void *dy, const void *x,
                                const int32_t *offsets, float *dw, uint32_t *err_word,
                                cudaStream_t stream)
{
    if (N == 0)  // no rows, and nothing the tensor maps could describe
        return cudaMemsetAsync(dw, 0, (size_t)E * M * K * sizeof(float), stream);
    cudaError_t st = cudaFuncSetAttribute(
        expert_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)W_SMEM);
    if (st != cudaSuccess)
        return st;
    CUtensorMap map_dy, map_x;
    st = encode_map(&map_dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy, 1, N, M, W_STEP, 64);
    if (st != cudaSuccess)
        return st;
    st = encode_map(&map_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, 1, N, K, W_STEP, 64);
    if (st != cudaSuccess)
        return st;
    const WgradArgs g = {N, M, K, E, (M + W_M - 1) / W_M, (K + W_K - 1) / W_K, offsets, dw,
                         err_word};
    const int64_t tiles = (int64_t)E * g.m_tiles * g.k_tiles;
    const int grid = (int)(tiles < sm_count() ? tiles : sm_count());
    return launch_pdl(expert_wgrad_kernel, dim3(grid), dim3(W_THREADS), W_SMEM, stream, map_dy,
                      map_x, g);
}

}  // namespace moe

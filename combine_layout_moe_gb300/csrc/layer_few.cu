// A whole mixture-of-experts layer for a few tokens (sm_103a), in two kernels.
//
//   out[t] = sum_e w[t,e] * W2_e ( silu(Wg_e x[t]) * (Wu_e x[t]) ),
//
// w[t,e] the sum of token t's weights over the slots that name e.  With few rows
// an expert the layer is a stream of weights: every chosen expert's are read
// once, at the rate of the HBM, and what is computed on the way has to keep up
// with it.  So a CTA's eight warps take 16 weight rows each (one mma tile), a
// producer warp keeps a ring of 128-byte-wide weight boxes and the matching piece
// of the activations in flight, and each warp multiplies its tile with all of the
// expert's tokens (mma.sync, tokens as columns in groups of eight).  The tile's
// sums stay in its warp: no exchange inside a product.  A tcgen05.mma would take
// at least 64 rows a tile and FP8 activations to match FP8 weights; here they stay
// bf16, and E4M3 weights widen to bf16 in registers (exactly).
//
// First kernel (UP): a tile is 8 gate rows and the 8 up rows of the same channels,
// so SwiGLU is a lane's own; h, weighted, goes to the workspace as two bf16 terms.
// The (expert, channel) range is cut evenly over the CTAs.  Second (DOWN): a tile
// is 16 output rows; a CTA takes up to eight tiles for a share of the experts and
// adds the experts up in shared memory, warp by warp; where experts are shared out,
// the last CTA of a group of rows adds the shares in a fixed order.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "tensormap.h"

namespace moe {

namespace {

constexpr int FEW_WARPS = 8;  // consumers
constexpr int FEW_THREADS = 32 * (FEW_WARPS + 1);
constexpr int FEW_MAX_STAGES = 16;
constexpr int FEW_TILE = 2048;  // 16 rows x 128 bytes
constexpr int FEW_W_BYTES = FEW_WARPS * FEW_TILE;
constexpr int FEW_MAX_SPLIT = 8;  // CTAs that may share the experts of a row group
constexpr size_t FEW_SMEM = 227 * 1024;

template <typename W>
struct FewType;
template <>
struct FewType<uint8_t> {
    static constexpr int KB = 128;   // inputs of a stage: 128 bytes of a weight row
    static constexpr int STEPS = 8;  // of K = 16
    static constexpr int WIDTH = 2;  // 128-byte pieces of an activation row
};
template <>
struct FewType<__nv_bfloat16> {
    static constexpr int KB = 64;
    static constexpr int STEPS = 4;
    static constexpr int WIDTH = 1;
};

struct FewShared {
    uint64_t full[FEW_MAX_STAGES], empty[FEW_MAX_STAGES];
    uint32_t tokens[2][MOE_MAX_EXPERTS];   // bit t: expert e is named by token t
    int ids[MOE_FEW_MAX_PAIRS];            // topk_idx
    int act[MOE_FEW_MAX_PAIRS];            // experts in use, by id
    int row0[MOE_FEW_MAX_PAIRS + 1];       // first row of each in h
    float w[MOE_FEW_MAX_PAIRS];            // weight of each row
    uint8_t token[MOE_FEW_MAX_PAIRS];      // token of each row
    int16_t pos[MOE_MAX_EXPERTS];          // place of e in act
    int active, longest, last;
    int failed;                            // a wait gave up
};

// Weights in boxes of 1, 2, 4 and 8 tiles' rows (UP: of one half, gate or up).
// Activations, UP: all T rows of x in act[0]; DOWN: 8, 16, 32 or 64 rows of h,
// both terms.
struct FewMaps {
    CUtensorMap w[4], act[4];
};

struct FewArgs {
    int T, k, H, I, E;
    const __nv_bfloat16 *x;  // UP: activations
    __nv_bfloat16 *h;        // [row][two terms][I]
    const int32_t *idx;
    const float *topk_w;
    const float *scales;
    float *parts;            // DOWN: [split][T][H]
    uint32_t *arrived;       // DOWN: per row group
    int groups;              // of `arrived`, that UP clears
    void *out;
    bool out_f32;
    uint32_t *err_word;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes 0 and 2, and bytes 1 and 3, of four E4M3 codes as bf16 pairs, exactly: the
// code's exponent and mantissa fields at the foot of bf16's exponent, then times
// 2^120, the difference of the biases (which also normalises subnormals).  The
// two NaN codes come out as 480; `seen` gathers them in its bytes' top bits.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &even, uint32_t &odd, uint32_t &seen)
{
    constexpr uint32_t S = 0x80008000u, F = 0x07f007f0u;
    const uint32_t up = 0x7b807b80u;  // 2^120 twice
    const uint32_t e = ((w << 8) & S) | ((w << 4) & F), o = (w & S) | ((w >> 4) & F);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(up));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(up));
    seen |= (w & 0x7f7f7f7fu) + 0x01010101u;
}

// Who names whom, in shared memory; called by the whole CTA.
__device__ void few_lists(FewShared &s, const FewArgs &g, bool weights, uint32_t *err_word)
{
    const int pairs = g.T * g.k;
    for (int e = threadIdx.x; e < g.E; e += FEW_THREADS)
        s.tokens[0][e] = s.tokens[1][e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += FEW_THREADS) {
        int e = g.idx[p];
        if (e < 0 || e >= g.E) {
            report(err_word, MOE_ERRBIT_BAD_INDEX);
            e = -1;
        } else {
            const int t = p / g.k;
            atomicOr(&s.tokens[t >> 5][e], 1u << (t & 31));
        }
        s.ids[p] = e;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int n = 0, rows = 0, longest = 0;
        for (int e0 = 0; e0 < g.E; e0 += 32) {
            const int e = e0 + lane;
            const int mine = e < g.E ? __popc(s.tokens[0][e]) + __popc(s.tokens[1][e]) : 0;
            const unsigned used = __ballot_sync(FULL_MASK, mine > 0);
            if (used == 0)
                continue;
            int sum = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(FULL_MASK, sum, d);
                if (lane >= d)
                    sum += v;
            }
            if (mine > 0) {
                const int at = n + __popc(used & lanemask_lt());
                s.act[at] = e;
                s.pos[e] = (int16_t)at;
                s.row0[at] = rows + sum - mine;
            }
            n += __popc(used);
            rows += __shfl_sync(FULL_MASK, sum, 31);
            longest = max(longest, (int)__reduce_max_sync(FULL_MASK, (unsigned)mine));
        }
        if (lane == 0) {
            s.failed = 0;
            s.row0[n] = rows;
            s.active = n;
            s.longest = longest;
        }
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += FEW_THREADS) {
        const int e = s.ids[p], t = p / g.k, first = t * g.k;
        if (e < 0)
            continue;
        bool again = false;  // an earlier slot of the token names the same expert
        for (int q = first; q < p; q++)
            again |= s.ids[q] == e;
        if (again)
            continue;
        const uint32_t lo = s.tokens[0][e], hi = s.tokens[1][e];
        const int below = t < 32 ? __popc(lo & ((1u << t) - 1))
                                 : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1));
        const int row = s.row0[s.pos[e]] + below;
        s.token[row] = (uint8_t)t;
        if (weights) {
            float w = 0.0f;
            for (int q = p; q < first + g.k; q++)
                if (s.ids[q] == e)
                    w += g.topk_w[q];
            s.w[row] = w;
        }
    }
    __syncthreads();
}

// The smallest of 8, 16, 32, 64 (0 .. 3) that holds n.
__device__ __forceinline__ int box_of(int n) { return n <= 8 ? 0 : n <= 16 ? 1 : n <= 32 ? 2 : 3; }

// A stretch of work: up to eight tiles of one expert, over all of its inputs.
struct Pass {
    int a, tile, tiles;
};

struct Work {
    // UP: [q, end) over (expert in use, group of 8 channels).  DOWN: [q, end) over
    // the experts of this CTA's share; `tile`, `tiles` its rows
    int64_t q, end;
    int per, tile, tiles, split, shares;
};

template <bool DOWN>
__device__ Work few_work(const FewShared &s, const FewArgs &g)
{
    Work w = {};
    const int grid = gridDim.x, b = blockIdx.x;
    if (!DOWN) {
        w.per = g.I / 8;
        const int64_t all = (int64_t)s.active * w.per;
        w.q = all * b / grid;
        w.end = all * (b + 1) / grid;
        return w;
    }
    // tiles a CTA takes, and shares of the experts: the fewest bytes for the
    // busiest CTA, and then the fewest shares
    const int all = (g.H + 15) / 16, experts = max(s.active, 1);
    int best = 0, shares = 1, cost = 0x7fffffff;
    for (int n = 1; n <= FEW_WARPS; n++) {
        const int groups = (all + n - 1) / n;
        const int sh = min(min(grid / groups, experts), FEW_MAX_SPLIT);
        const int rounds = sh >= 1 ? 1 : (groups + grid - 1) / grid;
        const int c = rounds * n * ((experts + max(sh, 1) - 1) / max(sh, 1));
        if (c < cost || (c == cost && max(sh, 1) < shares)) {
            cost = c;
            best = n;
            shares = max(sh, 1);
        }
    }
    w.per = best;
    w.shares = shares;
    return w;
}

template <bool DOWN>
__device__ __forceinline__ Pass next_pass(Work &w)
{
    Pass p;
    if (DOWN) {
        p.a = (int)w.q++;
        p.tile = w.tile;
        p.tiles = w.tiles;
    } else {
        p.a = (int)(w.q / w.per);
        p.tile = (int)(w.q - (int64_t)p.a * w.per);
        const int left = (int)min((int64_t)(w.per - p.tile), w.end - w.q);
        // equal passes
        p.tiles = (left + (left + FEW_WARPS - 1) / FEW_WARPS - 1) /
                  ((left + FEW_WARPS - 1) / FEW_WARPS);
        w.q += p.tiles;
    }
    return p;
}

// W: the weights' type.  NG: groups of eight tokens that an expert may have.
template <typename W, int NG, bool DOWN>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    few_kernel(const __grid_constant__ FewMaps maps, const FewArgs g)
{
    using TY = FewType<W>;
    constexpr bool FP8 = sizeof(W) == 1;
    constexpr int TERMS = DOWN ? 2 : 1;
    // a tile's rows 0-7, and from them to rows 8-15
    constexpr int TILE_STEP = DOWN ? 2048 : 1024, HALF_STEP = DOWN ? 1024 : FEW_WARPS * 1024;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~(uintptr_t)1023);
    uint8_t *top = raw + FEW_SMEM;
    FewShared &sh = *reinterpret_cast<FewShared *>(top - sizeof(FewShared));
    // DOWN: sums of 16 outputs x T tokens for each warp
    float *sums = reinterpret_cast<float *>(top - sizeof(FewShared)) - FEW_WARPS * 16 * g.T;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int K = DOWN ? g.I : g.H;
    const int blocks = (K + TY::KB - 1) / TY::KB;

    wait_prior_grid();
    allow_next_grid();
    if (threadIdx.x == 0) {
        for (int i = 0; i < FEW_MAX_STAGES; i++) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), FEW_WARPS);
        }
        mbar_fence_init();
    }
    if (!DOWN) {  // the second kernel's counters
        const int i = blockIdx.x * FEW_THREADS + threadIdx.x;
        if (i < g.groups)
            g.arrived[i] = 0;
    }
    few_lists(sh, g, !DOWN, !DOWN && blockIdx.x == 0 ? g.err_word : nullptr);

    // rows of a stage's activations: all tokens of x, or the most that an expert has
    const int act_rows = DOWN ? 16 << box_of(sh.longest) : (g.T + 7) & ~7;
    const Work whole = few_work<DOWN>(sh, g);
    const uint8_t *ring_end = DOWN ? reinterpret_cast<uint8_t *>(sums)
                                   : top - sizeof(FewShared);
    const int ring_bytes = (int)(ring_end - ring);
    // DOWN: a CTA of few tiles splits the inputs over its warps as well, `slices`
    // blocks a stage (as long as four stages fit); the slices' sums meet at the end
    const int slice_w = DOWN ? whole.per * FEW_TILE : FEW_W_BYTES;
    const int slice_bytes = slice_w + TY::WIDTH * act_rows * 128;
    const int slices =
        DOWN ? max(min(FEW_WARPS / whole.per, ring_bytes / (4 * slice_bytes)), 1) : 1;
    const int stage_bytes = slices * slice_bytes;
    // at least three: a slice is 48 KB at most, and the ring has 170
    const int stages = min(ring_bytes / stage_bytes, FEW_MAX_STAGES);
    const int row_tiles = (g.H + 15) / 16;
    const int groups = DOWN ? (row_tiles + whole.per - 1) / whole.per : 0;
    const int rounds = DOWN ? groups * whole.shares : (int)gridDim.x;
    int s = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;  // false once one of this warp's waits gave up

    for (int job = blockIdx.x; ok && job < rounds; job += gridDim.x) {
        Work work = whole;
        if (DOWN) {
            const int group = job / whole.shares;
            work.split = job - group * whole.shares;
            work.tile = group * whole.per;
            work.tiles = min(whole.per, row_tiles - work.tile);
            work.q = (int64_t)sh.active * work.split / whole.shares;
            work.end = (int64_t)sh.active * (work.split + 1) / whole.shares;
        }
        if (warp == FEW_WARPS) {
            while (ok && work.q < work.end) {
                const Pass p = next_pass<DOWN>(work);
                const int e = sh.act[p.a], row0 = sh.row0[p.a], n = sh.row0[p.a + 1] - row0;
                const int box = box_of(n);
                const int rows = DOWN ? 16 << box : g.T;  // of the activations' box
                const int row = DOWN ? 2 * row0 : 0;
                const CUtensorMap *act = &maps.act[DOWN ? box : 0];
                const int wrow = p.tile * (DOWN ? 16 : 8);
                for (int b0 = 0; b0 < blocks; b0 += slices) {
                    if (!(ok = warp_wait(smem_addr(&sh.empty[s]), phase ^ 1)))
                        break;
                    const uint32_t bar = smem_addr(&sh.full[s]);
                    uint32_t at = smem_addr(ring) + s * stage_bytes;
                    const int end = min(b0 + slices, blocks);
                    if (elect_one()) {
                        mbar_arrive_expect_tx(
                            bar, (end - b0) * (p.tiles * FEW_TILE + TY::WIDTH * rows * 128));
                        for (int b = b0; b < end; b++, at += slice_bytes) {
                            int done = 0;  // tiles, in boxes of falling size
#pragma unroll
                            for (int i = 3; i >= 0; i--) {
                                if (!(p.tiles >> i & 1))
                                    continue;
                                const int r = wrow + done * (DOWN ? 16 : 8);
                                tensor_g2s(at + done * TILE_STEP, &maps.w[i], b * TY::KB, r, e,
                                           bar);
                                if (!DOWN)
                                    tensor_g2s(at + HALF_STEP + done * TILE_STEP, &maps.w[i],
                                               b * TY::KB, g.I + r, e, bar);
                                done += 1 << i;
                            }
#pragma unroll
                            for (int i = 0; i < TY::WIDTH; i++)
                                tensor_g2s(at + slice_w + i * act_rows * 128, act,
                                           b * TY::KB + i * 64, row, 0, bar);
                        }
                    }
                    issued++;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            continue;
        }

        if (DOWN) {
            named_barrier(1, 32 * FEW_WARPS);  // the job before has been read
            for (int i = lane; i < 16 * g.T; i += 32)
                sums[warp * 16 * g.T + i] = 0.0f;
            __syncwarp();
        }
        const int r8 = lane >> 2, c4 = lane & 3;  // this lane's row (and row + 8) and columns
        while (ok && work.q < work.end) {
            const Pass p = next_pass<DOWN>(work);
            const int e = sh.act[p.a], row0 = sh.row0[p.a], n = sh.row0[p.a + 1] - row0;
            const int slice = DOWN ? warp / whole.per : 0;
            const int in_pass = DOWN ? warp - slice * whole.per : warp;
            const bool busy = slice < slices && in_pass < p.tiles;
            const int tile = p.tile + in_pass;
            const float *s_lo = nullptr, *s_hi = nullptr;  // of rows 0-7 and 8-15
            float v_lo = 0.0f, v_hi = 0.0f;
            if (FP8 && busy) {
                if (DOWN) {
                    s_lo = g.scales + ((int64_t)e * (g.H / 128) + tile / 8) * blocks;
                    s_hi = s_lo;
                } else {
                    s_lo = g.scales + ((int64_t)e * (2 * g.I / 128) + tile / 16) * blocks;
                    s_hi = s_lo + (int64_t)(g.I / 128) * blocks;
                }
            }
            float acc[NG][4];
#pragma unroll
            for (int i = 0; i < NG; i++)
                acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
            // where in a stage the activations of this lane's column begin (E4M3
            // weights: column r8; bf16: row lane % 8 of ldmatrix)
            uint32_t col_row[NG];
#pragma unroll
            for (int i = 0; i < NG; i++) {
                const int col = i * 8 + (FP8 ? r8 : lane & 7);
                col_row[i] = DOWN ? 2 * col : col < n ? sh.token[row0 + col] : 0;
            }
            uint32_t nan_lo = 0, nan_hi = 0;
            for (int b0 = 0, mine = 0; b0 < blocks; b0 += slices, mine++) {
                const int b = b0 + slice;
                if (FP8 && busy && (mine & 31) == 0) {  // of the next 32 blocks, one a lane
                    const int at = min(b + lane * slices, blocks - 1);
                    v_lo = s_lo[at];
                    v_hi = s_hi[at];
                }
                if (!(ok = warp_wait(smem_addr(&sh.full[s]), phase)))
                    break;
                if (busy && b < blocks) {
                    const uint32_t at =
                        smem_addr(ring) + s * stage_bytes + slice * slice_bytes;
                    const uint32_t wt = at + in_pass * TILE_STEP + ((lane >> 3) & 1) * HALF_STEP +
                                        (lane & 7) * 128;
                    uint32_t a[TY::STEPS][4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        uint32_t v[4];  // rows 0-7 and 8-15 of 16-byte pieces 2j and 2j + 1
                        ldsm4(wt + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4), v);
                        if constexpr (FP8) {
                            widen(v[0], a[2 * j][0], a[2 * j][2], nan_lo);
                            widen(v[1], a[2 * j][1], a[2 * j][3], nan_hi);
                            widen(v[2], a[2 * j + 1][0], a[2 * j + 1][2], nan_lo);
                            widen(v[3], a[2 * j + 1][1], a[2 * j + 1][3], nan_hi);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                a[j][i] = v[i];
                        }
                    }
                    float f_lo = 1.0f, f_hi = 1.0f;
                    if (FP8) {
                        f_lo = __shfl_sync(FULL_MASK, v_lo, mine & 31);
                        f_hi = __shfl_sync(FULL_MASK, v_hi, mine & 31);
                    }
#pragma unroll
                    for (int grp = 0; grp < NG; grp++) {
                        if (grp * 8 < n) {
                            float part[2 * TERMS][4] = {};  // sums that do not wait for each other
#pragma unroll
                            for (int term = 0; term < TERMS; term++) {
                                const uint32_t r = col_row[grp] + term;
                                const uint32_t row = at + slice_w + r * 128;
                                if constexpr (FP8) {
                                    const uint32_t in = (c4 & 1) * 8;
#pragma unroll
                                    for (int j = 0; j < TY::STEPS; j++) {
                                        const uint2 v = lds64(
                                            row + (j >> 2) * act_rows * 128 + in +
                                            ((((j & 3) * 2 + (c4 >> 1)) ^ (r & 7)) << 4));
                                        mma16816(part[2 * term + (j & 1)], a[j], __byte_perm(v.x, v.y, 0x5410),
                                                 __byte_perm(v.x, v.y, 0x7632));
                                    }
                                } else {
#pragma unroll
                                    for (int j = 0; j < TY::STEPS; j += 2) {
                                        uint32_t v[4];
                                        ldsm4(row + (((j * 2 + (lane >> 3)) ^ (r & 7)) << 4), v);
                                        mma16816(part[2 * term], a[j], v[0], v[1]);
                                        mma16816(part[2 * term + 1], a[j + 1], v[2], v[3]);
                                    }
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                float v = part[0][i] + part[1][i];
                                if (DOWN)
                                    v += part[2 * TERMS - 2][i] + part[2 * TERMS - 1][i];
                                acc[grp][i] = fmaf(v, i < 2 ? f_lo : f_hi, acc[grp][i]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.empty[s]));
                if (++s == stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (!ok)
                break;
            if (!busy)
                continue;
            if (FP8) {  // a NaN code of a row makes the row NaN
                nan_lo |= __shfl_xor_sync(FULL_MASK, nan_lo, 1);
                nan_lo |= __shfl_xor_sync(FULL_MASK, nan_lo, 2);
                nan_hi |= __shfl_xor_sync(FULL_MASK, nan_hi, 1);
                nan_hi |= __shfl_xor_sync(FULL_MASK, nan_hi, 2);
                const float bad = __int_as_float(0x7fffffff);
#pragma unroll
                for (int i = 0; i < NG; i++) {
                    if (nan_lo & 0x80808080u)
                        acc[i][0] = acc[i][1] = bad;
                    if (nan_hi & 0x80808080u)
                        acc[i][2] = acc[i][3] = bad;
                }
            }
#pragma unroll
            for (int grp = 0; grp < NG; grp++) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int col = grp * 8 + c4 * 2 + i;
                    if (col >= n)
                        continue;
                    if (DOWN) {
                        float *to = sums + (warp * g.T + sh.token[row0 + col]) * 16 + r8;
                        to[0] += acc[grp][i];
                        to[8] += acc[grp][2 + i];
                    } else {
                        const float gate = acc[grp][i];
                        const float v = gate / (1.0f + expf(-gate)) * acc[grp][2 + i] *
                                        sh.w[row0 + col];
                        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                        const float rest = v - __bfloat162float(hi);  // NaN of an infinite v
                        const __nv_bfloat16 lo =
                            __float2bfloat16_rn(fabsf(rest) < 3.0e38f ? rest : 0.0f);
                        __nv_bfloat16 *to = g.h + (int64_t)(row0 + col) * 2 * g.I + tile * 8 + r8;
                        to[0] = hi;
                        to[g.I] = lo;
                    }
                }
            }
        }

        if (DOWN) {
            if (!ok)
                sh.failed = 1;
            named_barrier(1, 32 * FEW_WARPS);  // every warp's sums are complete
            if (sh.failed) {                   // and no warp waits for one that has left
                ok = false;
                continue;
            }
            // the slices of a tile, added up by its first warp
            const int o = (work.tile + warp) * 16 + (lane & 15);
            const bool mine = warp < work.tiles && o < g.H;
            float *tile_sums = sums + warp * 16 * g.T + (lane & 15);
            if (mine)
                for (int t = lane >> 4; t < g.T; t += 2)
                    for (int i = 1; i < slices; i++)
                        tile_sums[t * 16] += tile_sums[(i * whole.per * g.T + t) * 16];
            if (whole.shares > 1) {
                const int64_t plane = (int64_t)g.T * g.H;
                if (mine)
                    for (int t = lane >> 4; t < g.T; t += 2)
                        __stcg(g.parts + work.split * plane + (int64_t)t * g.H + o,
                               tile_sums[t * 16]);
                __threadfence();
                named_barrier(1, 32 * FEW_WARPS);
                if (threadIdx.x == 0)
                    sh.last = atomicAdd(&g.arrived[job / whole.shares], 1u) ==
                              (unsigned)whole.shares - 1;
                named_barrier(1, 32 * FEW_WARPS);
                if (!sh.last)
                    continue;
                __threadfence();
                if (mine)
                    for (int t = lane >> 4; t < g.T; t += 2) {
                        float v = 0.0f;
                        for (int i = 0; i < whole.shares; i++)
                            v += __ldcg(g.parts + i * plane + (int64_t)t * g.H + o);
                        tile_sums[t * 16] = v;
                    }
            }
            if (mine)
                for (int t = lane >> 4; t < g.T; t += 2) {
                    const int64_t at = (int64_t)t * g.H + o;
                    if (g.out_f32)
                        static_cast<float *>(g.out)[at] = tile_sums[t * 16];
                    else
                        static_cast<__nv_bfloat16 *>(g.out)[at] =
                            __float2bfloat16_rn(tile_sums[t * 16]);
                }
        }
    }
    if (warp == FEW_WARPS)  // copies still in flight land before the CTA may end
        for (int64_t i = issued > stages ? issued - stages : 0; i < issued; i++)
            ok = warp_wait(smem_addr(&sh.full[i % stages]), (i / stages) & 1) && ok;
    if (!ok)
        report(g.err_word, MOE_ERRBIT_TIMEOUT);
}

template <typename W, int NG, bool DOWN>
cudaError_t few(const FewMaps &maps, const FewArgs &g, cudaStream_t stream)
{
    auto *kernel = few_kernel<W, NG, DOWN>;
    const cudaError_t st = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FEW_SMEM);
    if (st != cudaSuccess)
        return st;
    return launch_pdl(kernel, dim3(sm_count()), dim3(FEW_THREADS), FEW_SMEM, stream, maps, g);
}

template <typename W, bool DOWN>
cudaError_t few_for(const FewArgs &g, const void *weights, cudaStream_t stream)
{
    constexpr CUtensorMapDataType type =
        sizeof(W) == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    FewMaps maps;
    cudaError_t st = cudaSuccess;
    for (int i = 0; i < 4 && st == cudaSuccess; i++)
        st = DOWN ? encode_map(&maps.w[i], type, sizeof(W), weights, g.E, g.H, g.I, 16 << i,
                               FewType<W>::KB)
                  : encode_map(&maps.w[i], type, sizeof(W), weights, g.E, 2 * (int64_t)g.I, g.H,
                               8 << i, FewType<W>::KB);
    for (int i = 0; i < (DOWN ? 4 : 1) && st == cudaSuccess; i++)
        st = DOWN ? encode_map(&maps.act[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.h, 1,
                               2 * (int64_t)g.T * g.k, g.I, 16 << i, 64)
                  : encode_map(&maps.act[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.x, 1, g.T,
                               g.H, g.T, 64);
    if (st != cudaSuccess)
        return st;
    // registers for the groups of eight that an expert can have at most
    if (g.T <= 8)
        return few<W, 1, DOWN>(maps, g, stream);
    if (g.T <= 16)
        return few<W, 2, DOWN>(maps, g, stream);
    if (g.T <= 32)
        return few<W, 4, DOWN>(maps, g, stream);
    return few<W, 8, DOWN>(maps, g, stream);
}

size_t counters(int H) { return ((size_t)(H + 15) / 16 * sizeof(uint32_t) + 255) & ~(size_t)255; }

size_t inner_bytes(int T, int k, int I)
{
    return ((size_t)T * k * 2 * I * sizeof(__nv_bfloat16) + 255) & ~(size_t)255;
}

template <typename W>
cudaError_t layer(FewArgs g, const void *w13, const float *s13, const void *w2, const float *s2,
                  cudaStream_t stream)
{
    g.scales = s13;
    const cudaError_t st = few_for<W, false>(g, w13, stream);
    if (st != cudaSuccess)
        return st;
    g.scales = s2;
    return few_for<W, true>(g, w2, stream);
}

}  // namespace

size_t layer_few_workspace_bytes(int T, int k, int H, int I)
{
    return counters(H) + inner_bytes(T, k, I) + (size_t)FEW_MAX_SPLIT * T * H * sizeof(float);
}

cudaError_t launch_layer_few(int T, int k, int H, int I, int E, const void *x, const int32_t *idx,
                             const float *topk_w, const void *w13, const float *s13,
                             const void *w2, const float *s2, bool fp8, void *out, bool out_f32,
                             void *workspace, uint32_t *err_word, cudaStream_t stream)
{
    if (T == 0)
        return cudaSuccess;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    FewArgs g = {};
    g.T = T;
    g.k = k;
    g.H = H;
    g.I = I;
    g.E = E;
    g.x = static_cast<const __nv_bfloat16 *>(x);
    g.idx = idx;
    g.topk_w = topk_w;
    g.arrived = reinterpret_cast<uint32_t *>(ws);
    g.groups = (H + 15) / 16;
    g.h = reinterpret_cast<__nv_bfloat16 *>(ws + counters(H));
    g.parts = reinterpret_cast<float *>(ws + counters(H) + inner_bytes(T, k, I));
    g.out = out;
    g.out_f32 = out_f32;
    g.err_word = err_word;
    return fp8 ? layer<uint8_t>(g, w13, s13, w2, s2, stream)
               : layer<__nv_bfloat16>(g, w13, nullptr, w2, nullptr, stream);
}

}  // namespace moe

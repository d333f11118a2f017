// fp4q_moe.cu -- a mixture-of-experts layer for a few tokens, in one kernel.
//
//   l = x Wr^T;  the top_k largest logits per token, softmax weights w;
//   h_p = silu(G_e x) * (U_e x)  for every pair p = (token, chosen expert e);
//   y   = sum over a token's pairs of w_p D_e h_p.
//
// With few tokens the layer is bound by the chosen experts' quantized weights,
// each read once, so everything else is arranged around one stream of them:
// one CTA per SM walks a static share of (group, 64-row tile) items, a group
// being up to 16 pairs of one expert, first of the gate/up matrices (32 rows
// of each), then of the down matrices.  Per CTA
//   warp 8 streams the items' weight rows through a ring of shared-memory
//     stages (TMA tiles of 32 rows x 128 bytes, 128-byte swizzle; the rows'
//     scale bytes by bulk copies).  It runs ahead of the layer's dependencies:
//     the first down tiles are on their way while h is still being computed;
//   warp 9 adds the pairs' activations to the stages, the down items' once all
//     of h is written;
//   warps 0-7 multiply: 4 quarters of the stage's k by 2 halves of its rows,
//     mma.sync m16n8k16 with the weights as the 16 rows and the pairs as the 8
//     columns; an item ends with the sum of the quarters.
// The weights are widened to fp16 in registers on their way from shared memory
// into the product; tcgen05.mma, whose operands lie in shared or tensor
// memory, would need them written back first, and with a few columns per
// expert the products are far below even the older instruction's rate.
//
// Activations enter the products as fp16 with one power of two per 32 values
// (the largest of the 32 in [2^12, 2^13)): bf16 inputs keep every bit down to
// 2^-25 of the largest, h keeps 11 bits where bf16 would keep 8.  Codes are
// exact in fp16, and so are NVFP4's products code x UE4M3 scale; E8M0 and fp32
// scales, and the powers of two, multiply the fp32 sums of 32 products.
//
// Sums across k are in a fixed order and a token's pairs are added in slot
// order, so results do not depend on timing.  The three points where all CTAs
// wait for one another (x and logits ready, h ready, pair results ready) count
// in the workspace; the launch is cooperative, so all CTAs are resident, and
// every wait is bounded: one that runs out records the library's fault word
// and its warp goes on without waiting, within bounds, to the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "fp4q_device.cuh"
#include "fp4q_launch.h"
#include "fp4q_tc.cuh"
#include "fp4q_tma.h"
#include "../../include/fp4q.h"

namespace fp4q {
namespace moe {

constexpr int MAX_TOKENS = FP4Q_MOE_MAX_TOKENS, MAX_TOPK = FP4Q_MOE_MAX_TOPK, MAX_EXPERTS = FP4Q_MOE_MAX_EXPERTS;
constexpr int MAX_PAIRS = MAX_TOKENS * MAX_TOPK;
constexpr int CONSUMERS = 8;                            // warps that multiply
constexpr int THREADS = 32 * (CONSUMERS + 2);
constexpr int GROUP = 16;                               // pairs per group, at most
constexpr int TILE = 64;                                // rows per item: two boxes of 32
constexpr int BOX_BYTES = 32 * 128;
constexpr int RING_BYTES = 190 * 1024;
constexpr int RED_BYTES = 18 * 1024;
constexpr int SMEM_BYTES = 1024 + RING_BYTES + RED_BYTES;
constexpr int MAX_STAGES = 12;
constexpr uint32_t kMaxSpins = 1u << 22;                // polls of a counter in global memory (about 1 us each)

enum Fmt : int { kMx = FP4Q_SCALE_E8M0, kNv = FP4Q_SCALE_UE4M3, kF8 = FP4Q_F8_BLOCK128 };

struct Matrix {
    CUtensorMap map;                // codes [experts * rows][bytes], boxes of 32 x 128 bytes
    const void* scales;
    const float* gscale;            // NVFP4: per expert (stride 1) or one (stride 0); nullptr: 1
    int gstride;
};

struct Control {                    // first bytes of the workspace: zero between calls
    unsigned int start, h_done, o_done, leaving;
    unsigned int pad[12];
};

struct Params {
    Matrix up, down;
    const uint16_t* x;              // bf16 [tokens][hidden]
    const uint16_t* router;         // bf16 [experts][hidden], or nullptr: ids and weights are given
    int* ids;                       // [tokens][top_k]
    float* weights;
    uint16_t* y;                    // bf16 [tokens][hidden]
    Control* ctl;
    float* logits;                  // [tokens][experts]
    __half* xs;                     // [tokens][hidden]
    float* xsc;                     // [tokens][hb]
    __half* h;                      // [pairs][inter]
    float* hsc;                     // [pairs][ib]
    float* o;                       // [pairs][hidden]
    int tokens, hidden, inter, experts, top_k, normalize;
    int hb, ib;                     // powers of two per row of xs and h, padded to a multiple of 4
    unsigned int* fault;
};

struct Plan {                       // what the CTA knows once the choices are made
    int groups;                     // (expert, up to GROUP pairs)
    int widest;                     // pairs of the largest group
    int stages, stage_bytes;
    uint32_t scales_at, acts_at, pows_at;       // offsets within a stage
    uint32_t act_pitch;
};

struct Shared {
    int id[MAX_PAIRS];
    float w[MAX_PAIRS];
    uint16_t list[MAX_PAIRS];                   // pairs by expert, then by number
    uint16_t first[MAX_EXPERTS + 1];            // an expert's pairs in the list
    uint16_t g_expert[MAX_PAIRS], g_first[MAX_PAIRS];
    uint8_t g_count[MAX_PAIRS];
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    Plan plan;
};
static_assert(sizeof(Shared) + SMEM_BYTES + 1024 <= 227 * 1024, "shared memory per CTA");

// ---------------------------------------------------------------- formats
template <int FMT>
struct Format {
    static constexpr bool f8 = FMT == kF8;
    static constexpr int CHUNKS = 2;                         // 128-byte chunks of a row per stage
    static constexpr int VALUES = CHUNKS * (f8 ? 128 : 256); // k per stage
    static constexpr int BLOCKS = VALUES / 32;
    static constexpr int SCALE_BYTES = FMT == kNv ? VALUES / 16 : FMT == kMx ? VALUES / 32 : 0;   // per row and stage
    static constexpr int SCALE_PITCH = SCALE_BYTES ? SCALE_BYTES + 16 : 0;
    static constexpr int ACT_PITCH = VALUES * 2 + 64;        // 64 mod 128: 16-byte reads by (pair, lane) hit all banks
    static constexpr int POW_PITCH = BLOCKS + 4;             // floats
};

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t ld_acquire(const unsigned int* p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Wait until `n` CTAs have counted; false (and the fault word set) when the wait runs out.
__device__ bool spin(const unsigned int* counter, unsigned int n, unsigned int* fault)
{
    for (uint32_t i = 0; i < kMaxSpins; ++i) {
        if (ld_acquire(counter) >= n) return true;
        if (i > 64u) __nanosleep(100);
    }
    atomicExch(fault, 1u);
    return false;
}

// 2^e such that the finite magnitude of fp32 pattern `bits` divided by it lies in [2^12, 2^13), and 2^-e.
__device__ __forceinline__ void power_of(uint32_t bits, float& pow, float& inv)
{
    int e = (int)(bits >> 23);
    if (e < 14) e = 14;                                      // 2^-e stays finite
    pow = as_f32((uint32_t)(e - 12) << 23);
    inv = as_f32((uint32_t)(254 - (e - 12)) << 23);
}

__device__ __forceinline__ uint32_t finite_bits(float v)
{
    const uint32_t b = as_u32(v) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- before the products
// x as fp16 and powers of two: four lanes per 32 values.
__device__ void convert_x(const Params& p)
{
    const int blocks = p.hidden / 32, total = p.tokens * blocks * 4;
    for (int i = blockIdx.x * THREADS + threadIdx.x; i < ((total + 31) & ~31); i += gridDim.x * THREADS) {
        const int u = i < total ? i : total - 1;             // whole warps take part in the maxima
        const int t = u / (blocks * 4), c = (u - t * blocks * 4) * 8;
        const uint4 w = *reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.hidden + c);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        float f[8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bf16_lo(v[j]);
            f[2 * j + 1] = bf16_hi(v[j]);
            m = max(m, max(finite_bits(f[2 * j]), finite_bits(f[2 * j + 1])));
        }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float pow, inv;
        power_of(m, pow, inv);
        if (i < total) {
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = f16x2(__fmul_rn(f[2 * j], inv), __fmul_rn(f[2 * j + 1], inv));
            *reinterpret_cast<uint4*>(p.xs + (int64_t)t * p.hidden + c) = make_uint4(r[0], r[1], r[2], r[3]);
            if ((u & 3) == 0) p.xsc[t * p.hb + c / 32] = pow;
        }
    }
}

// Logits: a warp per (expert, up to 8 tokens), fp32 products and sums.
__device__ void route_logits(const Params& p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.tokens + 7) / 8, tasks = p.experts * per;
    for (int task = warp * gridDim.x + blockIdx.x; task < tasks; task += gridDim.x * (THREADS / 32)) {
        const int e = task / per, t0 = (task - e * per) * 8, nt = min(8, p.tokens - t0);
        const uint16_t* r = p.router + (int64_t)e * p.hidden;
        const uint16_t* x = p.x + (int64_t)t0 * p.hidden;
        float s[8] = {};
#pragma unroll 2
        for (int c = lane * 8; c < p.hidden; c += 256) {
            const uint4 a = *reinterpret_cast<const uint4*>(r + c);
            const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (t >= nt) break;
                const uint4 b = *reinterpret_cast<const uint4*>(x + (int64_t)t * p.hidden + c);
                const uint32_t bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[t] = __fmaf_rn(bf16_lo(av[j]), bf16_lo(bv[j]), s[t]);
                    s[t] = __fmaf_rn(bf16_hi(av[j]), bf16_hi(bv[j]), s[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t >= nt) break;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s[t] += __shfl_xor_sync(0xffffffffu, s[t], d);
            if (lane == 0) p.logits[(t0 + t) * p.experts + e] = s[t];
        }
    }
}

// An order of fp32 values in which NaN is the largest: larger pattern, larger value.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = as_u32(v);
    if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// The top_k experts of every token and their weights, a warp per token.
__device__ void choose(const Params& p, Shared& sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int PER = MAX_EXPERTS / 32;
    for (int t = warp; t < p.tokens; t += THREADS / 32) {
        float v[PER];
        uint32_t key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            key[j] = 0;
            const int e = lane + 32 * j;
            if (32 * j < p.experts && e < p.experts) {
                v[j] = __ldcg(p.logits + t * p.experts + e);
                key[j] = ordered(v[j]);                       // at least 0x007fffff: 0 marks what is gone
            }
        }
        float sum_all = 0.0f, peak = 0.0f, mine = 0.0f;
        int chosen = -1;
        for (int k = 0; k < p.top_k; ++k) {
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (32 * j < p.experts) best = max(best, key[j]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            uint32_t at = 0xffffffffu;                        // the first expert that has it
#pragma unroll
            for (int j = PER - 1; j >= 0; --j)
                if (32 * j < p.experts && key[j] == top) at = (uint32_t)(lane + 32 * j);
            at = __reduce_min_sync(0xffffffffu, at);
            float val = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (32 * j < p.experts && (int)at == lane + 32 * j) {
                    val = v[j];
                    key[j] = 0;
                }
            val = __shfl_sync(0xffffffffu, val, at & 31);
            if (k == 0) {
                peak = val;
                if (!p.normalize) {
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (lane + 32 * j < p.experts) sum_all += expf(v[j] - peak);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) sum_all += __shfl_xor_sync(0xffffffffu, sum_all, d);
                }
            }
            if (lane == k) {
                chosen = (int)at;
                mine = expf(val - peak);
            }
        }
        float below = mine;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
        if (!p.normalize) below = sum_all;
        if (lane < p.top_k) {
            const float w = __fdiv_rn(mine, below);
            sh.id[t * p.top_k + lane] = chosen;
            sh.w[t * p.top_k + lane] = w;
            if (blockIdx.x == 0) {
                p.ids[t * p.top_k + lane] = chosen;
                p.weights[t * p.top_k + lane] = w;
            }
        }
    }
}

// The pairs by expert, the groups, and the shape of a stage.
template <int FMT>
__device__ void make_plan(const Params& p, Shared& sh)
{
    using F = Format<FMT>;
    const int pairs = p.tokens * p.top_k, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.experts; e += THREADS) {
        int n = 0;
        for (int i = 0; i < pairs; ++i) n += sh.id[i] == e;
        sh.first[e + 1] = (uint16_t)n;                        // counts; summed below
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int total = 0, groups = 0, widest = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.experts ? sh.first[e + 1] : 0;
            const int ng = (n + GROUP - 1) / GROUP;
            int sn = n, sg = ng;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sn, d), b = __shfl_up_sync(0xffffffffu, sg, d);
                if (lane >= d) sn += a, sg += b;
            }
            const int at = total + sn - n;
            for (int i = 0; i < ng; ++i) {
                const int g = groups + sg - ng + i, c = min(GROUP, n - i * GROUP);
                sh.g_expert[g] = (uint16_t)e;
                sh.g_first[g] = (uint16_t)(at + i * GROUP);
                sh.g_count[g] = (uint8_t)c;
            }
            widest = max(widest, min(GROUP, n));
            __syncwarp();
            if (e < p.experts) sh.first[e] = (uint16_t)at;
            total += __shfl_sync(0xffffffffu, sn, 31);
            groups += __shfl_sync(0xffffffffu, sg, 31);
            // the next 32 counts start at first[e0 + 33]; first[e0 + 32] is overwritten by them only
            __syncwarp();
        }
        widest = __reduce_max_sync(0xffffffffu, widest);
        if (lane == 0) {
            Plan& q = sh.plan;
            q.groups = groups;
            q.widest = widest;
            q.act_pitch = F::ACT_PITCH;
            q.scales_at = F::CHUNKS * 2 * BOX_BYTES;
            q.acts_at = q.scales_at + TILE * F::SCALE_PITCH;
            const int columns = widest > 8 ? 16 : 8;          // what the products read; those past `widest` are not copied
            q.pows_at = q.acts_at + columns * F::ACT_PITCH;
            q.stage_bytes = (int)((q.pows_at + columns * F::POW_PITCH * 4 + 1023u) & ~1023u);
            q.stages = min(MAX_STAGES, RING_BYTES / q.stage_bytes);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += THREADS) {
        int at = sh.first[e];
        for (int i = 0; i < pairs; ++i)
            if (sh.id[i] == e) sh.list[at++] = (uint16_t)i;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- the stream
// One phase of the layer: its matrices, its sizes, and this CTA's items.
struct Phase {
    const Matrix* m;
    int k;                          // values per row
    int tiles;                      // items per group
    int first, items;               // this CTA's items: first, first + gridDim.x, ... below items
    int rows;                       // rows per expert
    int second;                     // rows from an item's first box to its second
    int step;                       // rows from one item to the next
};

__device__ __forceinline__ Phase phase_of(const Params& p, const Plan& q, int which)
{
    Phase f;
    const int up_items = q.groups * (p.inter / 32);
    if (which == 0) {
        f.m = &p.up;
        f.k = p.hidden;
        f.tiles = p.inter / 32;
        f.first = blockIdx.x;
        f.items = up_items;
        f.rows = 2 * p.inter;
        f.second = p.inter;
        f.step = 32;
    } else {
        f.m = &p.down;
        f.k = p.inter;
        f.tiles = (p.hidden + TILE - 1) / TILE;
        // the CTAs that had one item fewer before come first
        f.first = (int)((blockIdx.x + gridDim.x - (unsigned)up_items % gridDim.x) % gridDim.x);
        f.items = q.groups * f.tiles;
        f.rows = p.hidden;
        f.second = 32;
        f.step = TILE;
    }
    return f;
}

template <int FMT>
__device__ void stream_weights(const Params& p, const Shared& sh, uint32_t ring)
{
    using F = Format<FMT>;
    const int lane = threadIdx.x & 31;
    const Plan& q = sh.plan;
    const uint32_t full0 = smem_of(sh.full), empty0 = smem_of(sh.empty);
    int s = 0;
    uint32_t ph = 1;
    for (int which = 0; which < 2; ++which) {
        const Phase f = phase_of(p, q, which);
        const int row_bytes = F::f8 ? f.k : f.k / 2, srb = FMT == kNv ? f.k / 16 : f.k / 32;
        for (int it = f.first; it < f.items; it += gridDim.x) {
            const int g = it / f.tiles, tile = it - g * f.tiles;
            const int row0 = sh.g_expert[g] * f.rows + tile * f.step;      // experts * rows is below 2^31
            for (int k0 = 0, b0 = 0; k0 < f.k; k0 += F::VALUES, b0 += F::CHUNKS * 128) {
                if (!__all_sync(0xffffffffu, tc::wait_phase(empty0 + 8u * s, ph, p.fault))) return;
                const uint32_t st = ring + (uint32_t)(s * q.stage_bytes), bar = full0 + 8u * s;
                const int chunks = min(F::CHUNKS, (row_bytes - b0 + 127) / 128);
                // the rows' scale bytes, widened to 16-byte boundaries (every matrix of scales ends on one)
                int64_t src[2] = {0, 0};
                uint32_t len[2] = {0, 0};
                if (FMT != kF8) {
                    const int want = min(F::SCALE_BYTES, srb - k0 / (FMT == kNv ? 16 : 32));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = tile * f.step + i * f.second + lane;
                        if (r >= f.rows) continue;                         // the second box may lie past the expert
                        const int64_t at = (int64_t)(row0 + i * f.second + lane) * srb + k0 / (FMT == kNv ? 16 : 32);
                        src[i] = at & ~(int64_t)15;
                        len[i] = (uint32_t)(((at + want + 15) & ~(int64_t)15) - src[i]);
                    }
                }
                const uint32_t scales = __reduce_add_sync(0xffffffffu, len[0] + len[1]);
                if (lane == 0) {
                    tc::mbar_expect_tx(bar, (uint32_t)(chunks * 2 * BOX_BYTES) + scales);
                    for (int c = 0; c < chunks; ++c) {
                        tc::tma_load_2d(st + (uint32_t)(c * 2 * BOX_BYTES), &f.m->map, b0 + c * 128, row0, bar);
                        tc::tma_load_2d(st + (uint32_t)(c * 2 * BOX_BYTES + BOX_BYTES), &f.m->map, b0 + c * 128,
                                        row0 + f.second, bar);
                    }
                }
                __syncwarp();
                if (FMT != kF8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (len[i])
                            tc::bulk_load(st + q.scales_at + (uint32_t)((32 * i + lane) * F::SCALE_PITCH),
                                          static_cast<const uint8_t*>(f.m->scales) + src[i], len[i], bar);
                }
                if (++s == q.stages) s = 0, ph ^= 1u;
            }
        }
    }
}

template <int FMT>
__device__ void stream_activations(const Params& p, const Shared& sh, uint32_t ring)
{
    using F = Format<FMT>;
    const int lane = threadIdx.x & 31;
    const Plan& q = sh.plan;
    const uint32_t full0 = smem_of(sh.full), empty0 = smem_of(sh.empty);
    int s = 0;
    uint32_t ph = 1;
    fence_async();                                          // x was converted by ordinary stores
    for (int which = 0; which < 2; ++which) {
        const Phase f = phase_of(p, q, which);
        if (which == 1 && f.first < f.items) {
            const bool ok = spin(&p.ctl->h_done, gridDim.x, p.fault);
            if (!__all_sync(0xffffffffu, ok)) return;
            fence_async();
        }
        const __half* acts = which == 0 ? p.xs : p.h;
        const float* pows = which == 0 ? p.xsc : p.hsc;
        const int pitch = which == 0 ? p.hb : p.ib;
        for (int it = f.first; it < f.items; it += gridDim.x) {
            const int g = it / f.tiles, n = sh.g_count[g];
            int row = 0;
            if (lane < n) {
                row = sh.list[sh.g_first[g] + lane];
                if (which == 0) row /= p.top_k;
            }
            for (int k0 = 0; k0 < f.k; k0 += F::VALUES) {
                if (!__all_sync(0xffffffffu, tc::wait_phase(empty0 + 8u * s, ph, p.fault))) return;
                const uint32_t st = ring + (uint32_t)(s * q.stage_bytes), bar = full0 + 8u * s;
                const int values = min(F::VALUES, f.k - k0);
                const uint32_t ab = (uint32_t)values * 2u, pb = (uint32_t)((values / 32 + 3) & ~3) * 4u;
                if (lane == 0) tc::mbar_expect_tx(bar, (uint32_t)n * (ab + pb));
                __syncwarp();
                if (lane < n) {
                    tc::bulk_load(st + q.acts_at + (uint32_t)(lane * F::ACT_PITCH), acts + (int64_t)row * f.k + k0, ab, bar);
                    tc::bulk_load(st + q.pows_at + (uint32_t)(lane * F::POW_PITCH * 4), pows + row * pitch + k0 / 32, pb, bar);
                }
                if (++s == q.stages) s = 0, ph ^= 1u;
            }
        }
    }
}

// ---------------------------------------------------------------- the products
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight E2M1 codes -> four f16 pairs, in order.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Eight E4M3 codes -> four f16 pairs, in order.
__device__ __forceinline__ void widen8(uint32_t lo, uint32_t hi, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "mov.b32 {a, b}, %4;\n\t"
        "mov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\t"
        "cvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(lo), "r"(hi));
}

// A UE4M3 byte as an f16 pair of equal halves.
__device__ __forceinline__ uint32_t ue4m3_pair(uint32_t c)
{
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(c));
    return __byte_perm(h, h, 0x1010);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a)
{
    uint32_t r;
    asm volatile("{\n\t.reg .u8 t;\n\tld.shared.u8 t, [%1];\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * CONSUMERS) : "memory"); }

// The consumer warps' part of one phase.  NT: tiles of 8 columns (pairs).
// Within 32 values of k, lane (g, t) = (lane / 4, lane % 4) holds values
// 8 t .. 8 t + 7 of rows g and g + 8 and of column g: the order of k inside a
// product is free as long as both operands share it.
template <int FMT, int NT>
__device__ void multiply(const Params& p, const Shared& sh, uint32_t ring, float* red, int which, int& s, uint32_t& ph,
                         bool& live)
{
    using F = Format<FMT>;
    constexpr int COLS = 8 * NT, PITCH = COLS + 1;           // of the partial sums, floats
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, half = warp >> 2;
    const Plan& q = sh.plan;
    const uint32_t full0 = smem_of(sh.full), empty0 = smem_of(sh.empty);
    const Phase f = phase_of(p, q, which);
    const int srb = FMT == kNv ? f.k / 16 : f.k / 32;
    int turn = 0;
    for (int it = f.first; it < f.items; it += gridDim.x) {
        const int grp = it / f.tiles, tile = it - grp * f.tiles;
        const int e = sh.g_expert[grp], n = sh.g_count[grp];
        const int row0 = e * f.rows + tile * f.step;
        const float* f8_scales = nullptr;                    // of this item's first box
        int f8_second = 0;
        if (FMT == kF8) {
            f8_scales = static_cast<const float*>(f.m->scales) + (int64_t)(row0 >> 7) * (f.k >> 7);
            f8_second = ((row0 + f.second) >> 7) * (f.k >> 7) - (row0 >> 7) * (f.k >> 7);
        }
        float acc[2][NT][4] = {};
        for (int k0 = 0; k0 < f.k; k0 += F::VALUES) {
            float fs[2][2];                                  // E4M3: two blocks of 128 per stage, two boxes
            if (FMT == kF8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int kb = (k0 >> 7) + i < (f.k >> 7) ? (k0 >> 7) + i : (f.k >> 7) - 1;
                    fs[0][i] = __ldg(f8_scales + kb);
                    fs[1][i] = __ldg(f8_scales + f8_second + kb);
                }
            }
            if (live) live = __all_sync(0xffffffffu, tc::wait_phase(full0 + 8u * s, ph, p.fault));
            const uint32_t st = ring + (uint32_t)(s * q.stage_bytes);
            const int blocks = min(F::BLOCKS, (f.k - k0) / 32);
            const uint32_t w0 = st + (uint32_t)((16 * half + g) * 128);
            uint32_t sc[2][2];                               // the scale bytes of this lane's four rows
            if (FMT != kF8) {
                const uint32_t at = (uint32_t)(k0 / (FMT == kNv ? 16 : 32));
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t row = (uint32_t)(row0 + i * f.second + 16 * half + 8 * r + g);
                        sc[i][r] = st + q.scales_at + (uint32_t)((32 * i + 16 * half + 8 * r + g) * F::SCALE_PITCH) +
                                   ((row * (uint32_t)srb + at) & 15u);
                    }
            }
            for (int b = quarter; b < blocks; b += 4) {
                uint32_t bf[NT][4];
                float pw[NT][2];
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const uint4 v = lds128(st + q.acts_at + (uint32_t)((8 * c + g) * F::ACT_PITCH + 64 * b + 16 * t));
                    bf[c][0] = v.x, bf[c][1] = v.y, bf[c][2] = v.z, bf[c][3] = v.w;
                    const uint32_t pa = st + q.pows_at + (uint32_t)(((8 * c + 2 * t) * F::POW_PITCH + b) * 4);
                    pw[c][0] = as_f32(lds32(pa));
                    pw[c][1] = as_f32(lds32(pa + F::POW_PITCH * 4));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {                // the two boxes
                    uint32_t a[2][4];
                    float rs[2] = {1.0f, 1.0f};
                    if (FMT == kF8) {
                        const uint32_t wa = w0 + (uint32_t)((b >> 2) * 2 * BOX_BYTES + i * BOX_BYTES) +
                                            ((uint32_t)((2 * (b & 3) + (t >> 1)) ^ g) << 4) + 8u * (t & 1);
                        const uint2 v0 = lds64(wa), v1 = lds64(wa + 1024u);
                        widen8(v0.x, v0.y, a[0]);
                        widen8(v1.x, v1.y, a[1]);
                        rs[0] = rs[1] = fs[i][b >> 2];
                    } else {
                        const uint32_t wa = w0 + (uint32_t)((b >> 3) * 2 * BOX_BYTES + i * BOX_BYTES) +
                                            ((uint32_t)((b & 7) ^ g) << 4) + 4u * t;
                        widen4(lds32(wa), a[0]);
                        widen4(lds32(wa + 1024u), a[1]);
                        if (FMT == kNv) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const uint32_t m = ue4m3_pair(lds8(sc[i][r] + 2u * b + (t >> 1)));
#pragma unroll
                                for (int j = 0; j < 4; ++j) a[r][j] = mul_f16x2(a[r][j], m);
                            }
                        } else {
                            rs[0] = e8m0_decode(lds8(sc[i][0] + b));
                            rs[1] = e8m0_decode(lds8(sc[i][1] + b));
                        }
                    }
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        float d[4] = {};
                        mma16(d, a[0][0], a[1][0], a[0][1], a[1][1], bf[c][0], bf[c][1]);
                        mma16(d, a[0][2], a[1][2], a[0][3], a[1][3], bf[c][2], bf[c][3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float m = FMT == kNv ? pw[c][j & 1] : __fmul_rn(rs[j >> 1], pw[c][j & 1]);
                            acc[i][c][j] = __fmaf_rn(d[j], m, acc[i][c][j]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty0 + 8u * s);
            if (++s == q.stages) s = 0, ph ^= 1u;
        }

        // the four quarters of k, added in order
        float* buf = red + (NT == 1 ? turn * (4 * TILE * PITCH) : 0);
        turn ^= 1;
        if (NT > 1) consumers_sync();                        // one buffer: the last item's readers are done
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    buf[(quarter * TILE + 32 * i + 16 * half + g + 8 * (j >> 1)) * PITCH + 8 * c + 2 * t + (j & 1)] =
                        acc[i][c][j];
        consumers_sync();
        const float gs = FMT == kNv && f.m->gscale ? __ldg(f.m->gscale + e * f.m->gstride) : 1.0f;
        const uint16_t* list = sh.list + sh.g_first[grp];
        if (which == 0) {
            // a warp per pair: 32 consecutive values of h share a power of two
            for (int c = warp; c < n; c += CONSUMERS) {
                float a = 0.0f, b = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a += buf[(k * TILE + lane) * PITCH + c];
                    b += buf[(k * TILE + 32 + lane) * PITCH + c];
                }
                a = __fmul_rn(a, gs);
                b = __fmul_rn(b, gs);
                const float v = __fmul_rn(__fdiv_rn(a, 1.0f + expf(-a)), b);
                float pow, inv;
                power_of(__reduce_max_sync(0xffffffffu, finite_bits(v)), pow, inv);
                const int64_t pair = list[c];
                p.h[pair * p.inter + tile * 32 + lane] = __float2half_rn(__fmul_rn(v, inv));
                if (lane == 0) p.hsc[pair * p.ib + tile] = pow;
            }
        } else {
            const int r = tid & (TILE - 1);
            if (tile * TILE + r < p.hidden)
                for (int c = tid / TILE; c < n; c += 32 * CONSUMERS / TILE) {
                    float a = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) a += buf[(k * TILE + r) * PITCH + c];
                    p.o[(int64_t)list[c] * p.hidden + tile * TILE + r] = __fmul_rn(a, gs);
                }
        }
    }
}

// All of this CTA's consumer warps have stored: count it.
__device__ __forceinline__ void consumers_count(unsigned int* counter)
{
    consumers_sync();
    if (threadIdx.x == 0) {
        __threadfence();
        fence_async();
        atomicAdd(counter, 1u);
    }
}

template <int FMT>
__global__ void __launch_bounds__(THREADS, 1) moe_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_moe[];
    __shared__ Shared sh;
    const uint32_t raw = smem_of(smem_moe), ring = (raw + 1023u) & ~1023u;
    float* red = reinterpret_cast<float*>(smem_moe + (ring - raw) + RING_BYTES);
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            tc::mbar_init(smem_of(&sh.full[i]), 2u);
            tc::mbar_init(smem_of(&sh.empty[i]), (uint32_t)CONSUMERS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    convert_x(p);
    if (p.router) route_logits(p);
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        fence_async();
        atomicAdd(&p.ctl->start, 1u);
        spin(&p.ctl->start, gridDim.x, p.fault);
    }
    __syncthreads();
    if (p.router) {
        choose(p, sh);
    } else {
        for (int i = threadIdx.x; i < p.tokens * p.top_k; i += THREADS) {
            sh.id[i] = p.ids[i];
            sh.w[i] = p.weights[i];
        }
    }
    __syncthreads();
    make_plan<FMT>(p, sh);

    if (warp < CONSUMERS) {
        int s = 0;
        uint32_t ph = 0;
        bool live = true;
        const bool narrow = sh.plan.widest <= 8;
        if (narrow)
            multiply<FMT, 1>(p, sh, ring, red, 0, s, ph, live);
        else
            multiply<FMT, 2>(p, sh, ring, red, 0, s, ph, live);
        consumers_count(&p.ctl->h_done);
        if (narrow)
            multiply<FMT, 1>(p, sh, ring, red, 1, s, ph, live);
        else
            multiply<FMT, 2>(p, sh, ring, red, 1, s, ph, live);
        consumers_count(&p.ctl->o_done);
    } else if (warp == CONSUMERS) {
        stream_weights<FMT>(p, sh, ring);
    } else {
        stream_activations<FMT>(p, sh, ring);
    }
    __syncthreads();
    if (threadIdx.x == 0) spin(&p.ctl->o_done, gridDim.x, p.fault);
    __syncthreads();

    // y: a token's pairs in slot order, four columns per thread
    const int quads = p.hidden / 4;
    for (int i = blockIdx.x * THREADS + threadIdx.x; i < p.tokens * quads; i += gridDim.x * THREADS) {
        const int t = i / quads, c = (i - t * quads) * 4;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < p.top_k; ++k) {
            const int pair = t * p.top_k + k;
            if ((unsigned)sh.id[pair] >= (unsigned)p.experts) continue;
            const float w = sh.w[pair];
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.o + (int64_t)pair * p.hidden + c));
            sum.x = __fmaf_rn(w, v.x, sum.x);
            sum.y = __fmaf_rn(w, v.y, sum.y);
            sum.z = __fmaf_rn(w, v.z, sum.z);
            sum.w = __fmaf_rn(w, v.w, sum.w);
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
        *reinterpret_cast<uint2*>(p.y + (int64_t)t * p.hidden + c) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (threadIdx.x == 0) {
        // the last CTA to get here leaves the counters as it found them
        if (atomicAdd(&p.ctl->leaving, 1u) == gridDim.x - 1) {
            p.ctl->start = p.ctl->h_done = p.ctl->o_done = 0u;
            __threadfence();
            p.ctl->leaving = 0u;
        }
    }
}

// ---------------------------------------------------------------- host
struct Layout {
    size_t logits, xs, xsc, h, hsc, o, total;
};

Layout layout(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k)
{
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    const size_t pairs = (size_t)(tokens * top_k);
    const size_t hb = (size_t)((hidden / 32 + 3) & ~(int64_t)3), ib = (size_t)((inter / 32 + 3) & ~(int64_t)3);
    Layout l;
    l.logits = 256;
    l.xs = l.logits + up((size_t)(tokens * experts) * 4);
    l.xsc = l.xs + up((size_t)(tokens * hidden) * 2);
    l.h = l.xsc + up((size_t)tokens * hb * 4);
    l.hsc = l.h + up(pairs * (size_t)inter * 2);
    l.o = l.hsc + up(pairs * ib * 4);
    l.total = l.o + up(pairs * (size_t)hidden * 4);
    return l;
}

int check(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k)
{
    if (tokens < 0 || hidden <= 0 || inter <= 0 || experts <= 0 || top_k <= 0) return FP4Q_ERR_SHAPE;
    if (tokens > MAX_TOKENS || experts > MAX_EXPERTS || top_k > MAX_TOPK || top_k > experts) return FP4Q_ERR_UNSUPPORTED;
    if (hidden > 65536 || inter > 65536) return FP4Q_ERR_UNSUPPORTED;
    return FP4Q_OK;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

template <int FMT>
int launch(Params& p, cudaStream_t s)
{
    const int grid = resident_ctas((const void*)moe_kernel<FMT>, SMEM_BYTES, THREADS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_kernel<FMT>, p) == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

}  // namespace moe
}  // namespace fp4q

extern "C" size_t fp4q_moe_workspace_size(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k)
{
    if (fp4q::moe::check(tokens, hidden, inter, experts, top_k) != FP4Q_OK) return 0;
    return fp4q::moe::layout(tokens, hidden, inter, experts, top_k).total;
}

extern "C" int fp4q_moe(const void* x, int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k,
                        const void* router, int normalize, int fmt, const fp4q_moe_matrix* up,
                        const fp4q_moe_matrix* down, int32_t* ids, float* weights, void* y, void* workspace,
                        size_t ws_bytes, void* stream)
{
    using namespace fp4q;
    using namespace fp4q::moe;
    int st = check(tokens, hidden, inter, experts, top_k);
    if (st) return st;
    if (fmt != kMx && fmt != kNv && fmt != kF8) return FP4Q_ERR_UNSUPPORTED;
    const int unit = fmt == kF8 ? 128 : 32;
    if (hidden % unit || inter % unit) return FP4Q_ERR_SHAPE;
    if (tokens == 0) return FP4Q_OK;
    if (!x || !up || !down || !ids || !weights || !y || !workspace) return FP4Q_ERR_NULL;
    if (!up->codes || !up->scales || !down->codes || !down->scales) return FP4Q_ERR_NULL;
    if (fmt != kNv && (up->gscale || down->gscale)) return FP4Q_ERR_UNSUPPORTED;
    for (const fp4q_moe_matrix* m : {up, down}) {
        if (m->gscale_stride != 0 && m->gscale_stride != 1) return FP4Q_ERR_UNSUPPORTED;
        if (misaligned(m->codes, 16) || misaligned(m->scales, 16) || (m->gscale && misaligned(m->gscale, 4)))
            return FP4Q_ERR_ALIGN;
    }
    if (misaligned(x, 16) || (router && misaligned(router, 16)) || misaligned(ids, 4) || misaligned(weights, 4) ||
        misaligned(y, 16) || misaligned(workspace, 16))
        return FP4Q_ERR_ALIGN;
    const Layout l = layout(tokens, hidden, inter, experts, top_k);
    if (ws_bytes < l.total) return FP4Q_ERR_WORKSPACE;

    Params p;
    memset(&p, 0, sizeof(p));
    const int64_t per_byte = fmt == kF8 ? 1 : 2;
    if (!make_byte_map(&p.up.map, up->codes, experts * 2 * inter, hidden / per_byte, 32) ||
        !make_byte_map(&p.down.map, down->codes, experts * hidden, inter / per_byte, 32))
        return FP4Q_ERR_CUDA;
    p.up.scales = up->scales;
    p.up.gscale = up->gscale;
    p.up.gstride = up->gscale_stride;
    p.down.scales = down->scales;
    p.down.gscale = down->gscale;
    p.down.gstride = down->gscale_stride;
    p.x = static_cast<const uint16_t*>(x);
    p.router = static_cast<const uint16_t*>(router);
    p.ids = ids;
    p.weights = weights;
    p.y = static_cast<uint16_t*>(y);
    char* ws = static_cast<char*>(workspace);
    p.ctl = reinterpret_cast<Control*>(ws);
    p.logits = reinterpret_cast<float*>(ws + l.logits);
    p.xs = reinterpret_cast<__half*>(ws + l.xs);
    p.xsc = reinterpret_cast<float*>(ws + l.xsc);
    p.h = reinterpret_cast<__half*>(ws + l.h);
    p.hsc = reinterpret_cast<float*>(ws + l.hsc);
    p.o = reinterpret_cast<float*>(ws + l.o);
    p.tokens = (int)tokens;
    p.hidden = (int)hidden;
    p.inter = (int)inter;
    p.experts = (int)experts;
    p.top_k = (int)top_k;
    p.normalize = normalize != 0;
    p.hb = (int)((hidden / 32 + 3) & ~(int64_t)3);
    p.ib = (int)((inter / 32 + 3) & ~(int64_t)3);
    p.fault = device_fault_word();
    if (!p.fault) return FP4Q_ERR_CUDA;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (fmt == kMx) return launch<kMx>(p, cs);
    if (fmt == kNv) return launch<kNv>(p, cs);
    return launch<kF8>(p, cs);
}

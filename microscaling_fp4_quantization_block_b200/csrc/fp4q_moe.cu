// fp4q_moe.cu -- a mixture-of-experts layer for a few tokens, in one kernel.
//
//   l = x Wr^T;  the top_k largest logits per token, softmax weights w;
//   h_p = silu(G_e x) * (U_e x)  for every pair p = (token, chosen expert e);
//   y   = sum over a token's pairs of w_p D_e h_p.
//
// With few tokens the layer is bound by the chosen experts' quantized weights,
// so everything else is arranged around one stream of them:
// one CTA per SM walks a static share of (group, 64-row tile) items, a group
// being up to 16 pairs of one expert (for which its weights are read once), first
// of the gate/up matrices (32 rows of each), then of the down matrices, two items
// at a time.  Each of the two
// streams has half of a ring of shared-memory stages and, of the CTA's warps,
//   one (16, 18) that fetches the items' weight rows (TMA tiles of 32 rows x 128
//     bytes, 128-byte swizzle), ahead of the layer's dependencies: the first
//     down tiles are on their way while h is still being computed;
//   one (17, 19) that adds the rows' scale bytes and the pairs' activations
//     (16-byte cp.async: as bulk copies of 32 bytes the scale bytes took 45 ns
//     each, one after the other, eight times the weights' time);
//   eight (0-7, 8-15) that multiply, 4 quarters of a stage's k by 2 halves of its
//     rows, mma.sync m16n8k16 with the weights as the 16 rows and the pairs as
//     the 8 columns;
//   two (20 and 21, 22 and 23) that add the four slices of k and finish the item
//     (silu, h; or the pairs' results) while the next one is multiplied.
// The weights are widened to fp16 in registers on their way from shared memory
// into the product.  tcgen05.mma takes its operands from shared or tensor memory:
// written back to shared memory the weights would cost it four times what the
// codes do; as an operand in tensor memory (tcgen05.st) they would not, a form
// that has not been built.  mma.sync reaches 690 multiply-adds a clock
// and SM here, 15 columns' worth at the rate HBM delivers FP4 weights, so groups
// of more than 8 pairs are near its bound.
//
// Measured (a loop of calls; the experts' bytes at the copy rate of 6.55 TB/s in
// brackets): 1 token, 8 of 64 NVFP4 experts of 2048 x 1024, 29 us (4.4): launch,
// router, choices and the three waits take 17 of them; 5 tokens over E4M3 experts
// 55 us (26); 23 tokens over 60 NVFP4 experts 62 us (24); 64 tokens over 128 MXFP4
// experts of 2048 x 768 127 us (48); over 64 NVFP4 experts of 5120 x 1792 314 us
// (152).  With logits in fp32 these took 28, 55, 62, 127 and 299, and then without
// the products 25, 51, 51, 95 and 215: what bounds the long calls is the products'
// instructions on top of the stream that the warps filling the stages sustain, and
// that stream carries, beside the weights, a group's activations for every item.
//
// Activations enter the products as fp16 under one power of two per row (the
// row's largest value in [2^7, 2^8)): bf16 inputs keep every bit down to 2^-24
// of the largest and are off by at most 2^-32 of it below that.  h is rounded to
// fp16 under a power of its own per 32 values, which keeps 11 significant bits
// where bf16 would keep 8, and brought to its row's power: exact down to 2^-21
// of the row's largest value, off by at most 2^-24 of it below.  Codes are exact
// in fp16, and so are NVFP4's products code x UE4M3 scale; E8M0 and fp32 scales
// multiply the fp32 sums of their blocks.
//
// Sums across k are in a fixed order and a token's pairs are added in slot
// order, so results depend neither on timing nor on the call's other tokens.  The points where all CTAs
// wait for one another (x and logits, choices, h, pair results) count
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
constexpr int STREAMS = 2;                              // items in work at the same time
constexpr int SET = 8;                                  // warps that multiply, per stream
constexpr int CONSUMERS = STREAMS * SET;
constexpr int SUM_WARPS = 2;                            // per stream: add an item's slices and write its results
constexpr int FIRST_COPY = CONSUMERS, FIRST_SUM = FIRST_COPY + 2 * STREAMS;    // per stream a warp for weights, one for the rest
constexpr int THREADS = 32 * (FIRST_SUM + STREAMS * SUM_WARPS);
constexpr int REGS_PRODUCTS = 96, REGS_OTHERS = 48;     // 512 x 96 + 256 x 48 = 768 x 80, the launch's registers
constexpr int GROUP = 16;                               // pairs per group, at most
constexpr int TILE = 64;                                // rows per item: two boxes of 32
constexpr int BOX_BYTES = 32 * 128;
constexpr int WEIGHT_BYTES = 2 * 2 * BOX_BYTES;         // per stage: two 128-byte chunks of two boxes
constexpr int SLICES = 4;                               // of k, per item
constexpr int RING_BYTES = 172 * 1024;
constexpr int RED_BYTES = 36 * 1024;                    // partial sums: per stream two buffers of 8 columns or one of 16
constexpr int SMEM_BYTES = 1024 + RING_BYTES + RED_BYTES;
constexpr int MAX_STAGES = 12;
constexpr int MIN_STAGES = 4;
constexpr uint32_t NONE = 0xffffu;
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
    double* logits;                 // [slices of k][tokens][experts]
    uint8_t* xs;                    // [tokens][xstages] records (Format::RECORD bytes)
    float* xpow;                    // [tokens]
    uint8_t* h;                     // [pairs][hstages] records
    unsigned int* hmax;             // [pairs]: pattern of the largest finite |h|
    float* o;                       // [pairs][hidden]
    int tokens, hidden, inter, experts, top_k, normalize;
    int xstages, hstages;           // stages of hidden and of inter values
    unsigned int* fault;
};

struct Plan {                       // what the CTA knows once the choices are made
    int groups;                     // (expert, up to GROUP pairs)
    int widest;                     // pairs of the largest group
    int buffers;                    // of partial sums per stream: two where no item has more than 8 columns
    int stages;                     // an even number: every other slot of the ring is a stream's
    uint32_t aux_bytes, acts_at, inverse_at;    // what a stage holds beside its weights: scale bytes, records, 1 / the rows' powers
};

struct Shared {
    uint16_t id[MAX_PAIRS];                     // NONE: no expert
    int count[MAX_EXPERTS];                     // pairs by expert
    float w[MAX_PAIRS];
    uint16_t list[MAX_PAIRS];                   // pairs by expert, then by number
    uint16_t first[MAX_EXPERTS + 1];            // an expert's pairs in the list
    uint16_t g_expert[MAX_PAIRS], g_first[MAX_PAIRS];
    uint8_t g_count[MAX_PAIRS];
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t summed[STREAMS][2], summable[STREAMS][2];      // a buffer of partial sums: free, complete
    Plan plan;
};
static_assert(sizeof(Shared) + SMEM_BYTES + 1024 <= 227 * 1024, "shared memory per CTA");

// ---------------------------------------------------------------- formats
template <int FMT>
struct Format {
    static constexpr bool f8 = FMT == kF8;
    static constexpr int CHUNKS = 2;                         // 128-byte chunks of a row per stage
    static constexpr int VALUES = CHUNKS * (f8 ? 128 : 256); // k per stage
    static constexpr int QUARTER = VALUES / 4;               // k per warp and stage: 64 bytes of a row
    static constexpr int BLOCKS = VALUES / 32;
    static constexpr int SCALE_BYTES = FMT == kNv ? VALUES / 16 : FMT == kMx ? VALUES / 32 : 0;   // per row and stage
    static constexpr int SCALE_PITCH = SCALE_BYTES ? SCALE_BYTES + 16 : 0;
    // A row's activations of one stage, as they are kept and copied: fp16 values (zeros past the row's end), then
    // the powers of two of its blocks of 32 (h only).  64 mod 128 bytes: 16-byte reads by (pair, lane) hit all banks.
    static constexpr int POWERS = VALUES * 2, RECORD = POWERS + 64;
    static constexpr int AUX_MOST = TILE * SCALE_PITCH + GROUP * (RECORD + 4);
    static_assert(MIN_STAGES * (WEIGHT_BYTES + AUX_MOST) <= RING_BYTES, "a ring of at least four stages");
};

// Where value i of a stage's activations is kept.  In the products a lane t of
// four holds 16 bytes of a row's 64-byte quarter: 32 E2M1 values (one block, or
// under E8M0 scales a quarter of each of four blocks) or 16 E4M3 values.  The
// activations are stored so that the lane's 16-byte pieces j of one quarter lie
// [j][t]: reads of one piece by the four lanes are consecutive.
template <int FMT>
__device__ __forceinline__ int place(int i)
{
    if (FMT == kNv) return (i & ~127) | ((i >> 3) & 3) << 5 | ((i >> 5) & 3) << 3 | (i & 7);
    if (FMT == kF8) return (i & ~63) | ((i >> 3) & 1) << 5 | ((i >> 4) & 3) << 3 | (i & 7);
    return i;
}

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t ld_acquire(const unsigned int* p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// What other threads stored, for this thread's bulk copies.
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

// 2^e such that the finite magnitude of fp32 pattern `bits` divided by it lies in [2^7, 2^8), and 2^-e.
__device__ __forceinline__ void power_of(uint32_t bits, float& pow, float& inv)
{
    int e = (int)(bits >> 23);
    if (e < 9) e = 9;                                        // 2^-e stays finite
    pow = as_f32((uint32_t)(e - 7) << 23);
    inv = as_f32((uint32_t)(254 - (e - 7)) << 23);
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
// x as fp16 under a power of two per row: a CTA per token.
template <int FMT>
__device__ void convert_x(const Params& p, unsigned int* part)
{
    using F = Format<FMT>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = blockIdx.x * THREADS + threadIdx.x; i < p.tokens * p.top_k; i += gridDim.x * THREADS) p.hmax[i] = 0u;
    for (int t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const uint16_t* x = p.x + (int64_t)t * p.hidden;
        uint32_t m = 0;
        for (int c = threadIdx.x * 8; c < p.hidden; c += THREADS * 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(x + c);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, max(finite_bits(bf16_lo(v[j])), finite_bits(bf16_hi(v[j]))));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) part[warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) m = max(m, part[i]);
        float pow, inv;
        power_of(m, pow, inv);
        if (threadIdx.x == 0) p.xpow[t] = pow;
        uint8_t* to = p.xs + (int64_t)t * p.xstages * F::RECORD;
        for (int c = threadIdx.x * 8; c < p.xstages * F::VALUES; c += THREADS * 8) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (c < p.hidden) w = *reinterpret_cast<const uint4*>(x + c);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = f16x2(__fmul_rn(bf16_lo(v[j]), inv), __fmul_rn(bf16_hi(v[j]), inv));
            *reinterpret_cast<uint4*>(to + c / F::VALUES * F::RECORD + 2 * place<FMT>(c % F::VALUES)) =
                make_uint4(r[0], r[1], r[2], r[3]);
        }
        __syncthreads();                                     // part is free again
    }
}

// Slices of k that the logits are summed in, so that there is work for every
// warp of the grid: at most 8, of at least 256 values.  The number of tokens
// does not enter, so that a token's logits do not depend on who else is there.
__device__ __forceinline__ int logit_slices(const Params& p)
{
    return max(1, min(min(8, p.hidden / 256), (int)gridDim.x * (THREADS / 32) / p.experts));
}

// The sums over the warp's lanes of COUNT values each, by halves: lane l ends up
// with value l / (32 / COUNT).  Whatever COUNT, a value's sum is the same tree.
template <int COUNT>
__device__ __forceinline__ double lane_sums(double (&v)[COUNT])
{
    const int lane = threadIdx.x & 31;
    int n = COUNT;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        if (n > 1) {
            n /= 2;
            const bool upper = (lane & d) != 0;
#pragma unroll
            for (int i = 0; i < COUNT / 2; ++i)
                if (i < n) {
                    const double mine = upper ? v[i + n] : v[i], other = upper ? v[i] : v[i + n];
                    v[i] = mine + __shfl_xor_sync(0xffffffffu, other, d);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
        }
    }
    return v[0];
}

// One task: E experts from e0 against N tokens from t0 (those past the last
// repeat it).  The sums are held in 64 bits, where a product of two bf16 values
// is exact: which of two nearly equal logits is the larger decides a token's
// experts, and fp32 sums of equal logits differ.
template <int E, int N>
__device__ __forceinline__ void logits_of(const Params& p, int e0, int t0, int from, int to, double* out)
{
    constexpr int W = E * N > 8 ? 4 : 8;                     // values of a row at a time: registers
    const int lane = threadIdx.x & 31, last_t = p.tokens - 1, last_e = p.experts - 1;
    double s[E * N] = {};
    for (int c0 = from + lane * 8; c0 < to; c0 += 256) {
#pragma unroll
        for (int c = c0; c < c0 + 8; c += W) {
            uint32_t a[E][W / 2], b[N][W / 2];
            auto load = [&](uint32_t (&v)[W / 2], const uint16_t* from_row) {
                if constexpr (W == 8) {
                    const uint4 u = *reinterpret_cast<const uint4*>(from_row + c);
                    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(from_row + c);
                    v[0] = u.x, v[1] = u.y;
                }
            };
#pragma unroll
            for (int e = 0; e < E; ++e) load(a[e], p.router + (int64_t)min(e0 + e, last_e) * p.hidden);
#pragma unroll
            for (int t = 0; t < N; ++t) load(b[t], p.x + (int64_t)min(t0 + t, last_t) * p.hidden);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                double av[E];
#pragma unroll
                for (int e = 0; e < E; ++e) av[e] = (double)(j & 1 ? bf16_hi(a[e][j / 2]) : bf16_lo(a[e][j / 2]));
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    const double bv = (double)(j & 1 ? bf16_hi(b[t][j / 2]) : bf16_lo(b[t][j / 2]));
#pragma unroll
                    for (int e = 0; e < E; ++e) s[e * N + t] = __fma_rn(av[e], bv, s[e * N + t]);
                }
            }
        }
    }
    const double sum = lane_sums<E * N>(s);
    constexpr int LANES = 32 / (E * N);                      // that hold the same sum
    const int i = lane / LANES, e = e0 + i / N, t = t0 + i % N;
    if (lane % LANES == 0 && e <= last_e && t <= last_t) out[t * p.experts + e] = sum;
}

// Logits: a warp per (expert, up to 8 tokens, slice of k), or two experts where
// that still gives every warp a task (x is widened to 64 bits half as often);
// the slices are added by their reader, in order.
__device__ void route_logits(const Params& p)
{
    const int warp = threadIdx.x >> 5, warps = (int)gridDim.x * (THREADS / 32);
    const int per = (p.tokens + 7) / 8, slices = logit_slices(p);
    const int step = ((p.hidden + slices - 1) / slices + 7) & ~7;
    const bool pairs = p.tokens > 4 && p.experts * per * slices > warps;
    const int tasks = (pairs ? (p.experts + 1) / 2 : p.experts) * per * slices;
    for (int task = warp * gridDim.x + blockIdx.x; task < tasks; task += warps) {
        const int u = task / slices, k = task - u * slices, e = u / per, t0 = (u - e * per) * 8;
        const int from = k * step, to = min(p.hidden, from + step);
        double* out = p.logits + (int64_t)k * p.tokens * p.experts;
        if (pairs)
            logits_of<2, 8>(p, 2 * e, t0, from, to, out);
        else if (p.tokens - t0 == 1)
            logits_of<1, 1>(p, e, t0, from, to, out);
        else if (p.tokens - t0 <= 4)
            logits_of<1, 4>(p, e, t0, from, to, out);
        else
            logits_of<1, 8>(p, e, t0, from, to, out);
    }
}

// An order of 64-bit values in which NaN is the largest: larger pattern, larger value.
typedef unsigned long long Key;
constexpr Key kNanKey = ~0ull;

__device__ __forceinline__ Key ordered(double v)
{
    const Key b = (Key)__double_as_longlong(v);
    if ((b & ~(1ull << 63)) > 0x7ff0000000000000ull) return kNanKey;
    return (b >> 63) ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ double from_ordered(Key k)
{
    return __longlong_as_double((long long)(k == kNanKey ? 0x7ff8000000000000ull : (k >> 63) ? k ^ (1ull << 63) : ~k));
}

__device__ __forceinline__ Key warp_max(Key k)
{
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    return (Key)hi << 32 | __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
}

// The top_k experts of every token and their weights, a warp per token; a lane holds PER experts.
template <int PER>
__device__ void choose(const Params& p, Shared& sh, int first, int step, bool tell)
{
    const int lane = threadIdx.x & 31, slices = logit_slices(p);
    for (int t = first; t < p.tokens; t += step) {
        Key key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 32 * j;
            double part[8], v = 0.0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                part[k] = e < p.experts && k < slices ? __ldcg(p.logits + ((int64_t)k * p.tokens + t) * p.experts + e) : 0.0;
#pragma unroll
            for (int k = 0; k < 8; ++k) v += part[k];
            key[j] = e < p.experts ? ordered(v) : 0u;         // an expert's is at least 2^52 - 1: 0 marks what is gone
        }
        Key best = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) best = max(best, key[j]);
        const double peak = from_ordered(warp_max(best));
        float below = 0.0f;
        if (!p.normalize) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 32 * j < p.experts) below += expf((float)(from_ordered(key[j]) - peak));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
        }
        float mine = 0.0f;
        uint32_t chosen = NONE;
        for (int k = 0; k < p.top_k; ++k) {
            const Key top = warp_max(best);
            uint32_t at = NONE;                               // the first expert that has it
#pragma unroll
            for (int j = PER - 1; j >= 0; --j)
                if (key[j] == top) at = (uint32_t)(lane + 32 * j);
            at = __reduce_min_sync(0xffffffffu, at);
            best = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (at == (uint32_t)(lane + 32 * j)) key[j] = 0;
                best = max(best, key[j]);
            }
            if (lane == k) {
                chosen = at;
                mine = expf((float)(from_ordered(top) - peak));
            }
        }
        if (p.normalize) {
            below = mine;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
        }
        if (lane < p.top_k) {
            const float w = __fdiv_rn(mine, below);
            sh.id[t * p.top_k + lane] = (uint16_t)chosen;
            sh.w[t * p.top_k + lane] = w;
            if (tell) {
                p.ids[t * p.top_k + lane] = (int)chosen;
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
    for (int e = threadIdx.x; e < p.experts; e += THREADS) sh.count[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += THREADS)
        if (sh.id[i] != NONE) atomicAdd(&sh.count[sh.id[i]], 1);
    __syncthreads();
    if (threadIdx.x < 32) {
        int total = 0, groups = 0, widest = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.experts ? sh.count[e] : 0;
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
            if (e < p.experts) sh.first[e] = (uint16_t)at;
            total += __shfl_sync(0xffffffffu, sn, 31);
            groups += __shfl_sync(0xffffffffu, sg, 31);
        }
        if (lane == 0) sh.first[p.experts] = (uint16_t)total;
        widest = __reduce_max_sync(0xffffffffu, widest);
        if (lane == 0) {
            Plan& q = sh.plan;
            q.groups = groups;
            q.widest = widest;
            q.buffers = widest > 8 ? 1 : 2;
            q.acts_at = TILE * F::SCALE_PITCH;
            q.inverse_at = q.acts_at + widest * F::RECORD;
            q.aux_bytes = (q.inverse_at + widest * 4 + 15u) & ~15u;
            q.stages = min(MAX_STAGES, (int)(RING_BYTES / (WEIGHT_BYTES + q.aux_bytes))) & ~1;
        }
    }
    __syncthreads();
    // Within a group the order of the pairs changes nothing; which group a pair
    // of a long list falls into must be the same in every CTA: by number.
    for (int i = threadIdx.x; i < pairs; i += THREADS) {
        const uint32_t e = sh.id[i];
        if (e != NONE && sh.first[e + 1] - sh.first[e] <= GROUP)
            sh.list[sh.first[e] + atomicSub(&sh.count[e], 1) - 1] = (uint16_t)i;
    }
    if (sh.plan.widest == GROUP) {
        for (int e = threadIdx.x >> 5; e < p.experts; e += THREADS / 32) {
            int at = sh.first[e];
            if (sh.first[e + 1] - at <= GROUP) continue;
            for (int i = lane; i < ((pairs + 31) & ~31); i += 32) {
                const bool mine = i < pairs && sh.id[i] == (uint32_t)e;
                const uint32_t all = __ballot_sync(0xffffffffu, mine);
                if (mine) sh.list[at + __popc(all & ((1u << lane) - 1u))] = (uint16_t)i;
                at += __popc(all);
            }
        }
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
    int hop_groups, hop_tiles;      // a stream's next item: so many groups and tiles on
};

// A stream's items of a phase, one after the other: every STREAMS-th of the CTA's.
struct Item {
    int left;                       // items, this one included
    int group, tile;

    __device__ __forceinline__ Item(const Phase& f, int stream)
    {
        const int first = f.first + stream * (int)gridDim.x, hop = STREAMS * (int)gridDim.x;
        left = first < f.items ? (f.items - first + hop - 1) / hop : 0;
        group = first / f.tiles;
        tile = first - group * f.tiles;
    }
    __device__ __forceinline__ void next(const Phase& f)
    {
        --left;
        group += f.hop_groups;
        tile += f.hop_tiles;
        if (tile >= f.tiles) tile -= f.tiles, ++group;
    }
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
    f.hop_groups = STREAMS * (int)gridDim.x / f.tiles;
    f.hop_tiles = STREAMS * (int)gridDim.x % f.tiles;
    return f;
}

// A place in a stream's sequence of stages.  The ring is even, so that a slot
// always belongs to the same stream: a barrier's parity tells a phase only from
// the one before it, so whoever waits for a slot must have seen each of its
// rounds.
struct Slots {
    uint32_t full0, empty0;
    int n, at;
    uint32_t phase;

    __device__ Slots(const Shared& sh, int stream)
        : full0(smem_of(sh.full)), empty0(smem_of(sh.empty)), n(sh.plan.stages), at(stream), phase(1u) {}
    __device__ __forceinline__ bool wait_empty(unsigned int* fault) const
    {
        return tc::wait_phase(empty0 + 8u * at, phase, fault);
    }
    __device__ __forceinline__ void next()
    {
        at += STREAMS;
        if (at >= n) at -= n, phase ^= 1u;
    }
};

// The weights, by one lane.
template <int FMT>
__device__ __forceinline__ void stream_weights(const Params& p, const Shared& sh, uint32_t ring, int stream)
{
    using F = Format<FMT>;
    Slots s(sh, stream);
    for (int which = 0; which < 2; ++which) {
        const Phase f = phase_of(p, sh.plan, which);
        const int row_bytes = F::f8 ? f.k : f.k / 2;
        for (Item it(f, stream); it.left > 0; it.next(f)) {
            const int row0 = sh.g_expert[it.group] * f.rows + it.tile * f.step;      // experts * rows is below 2^31
            for (int b0 = 0; b0 < row_bytes; b0 += F::CHUNKS * 128) {
                if (!s.wait_empty(p.fault)) return;
                const uint32_t st = ring + (uint32_t)(s.at * WEIGHT_BYTES), bar = s.full0 + 8u * s.at;
                const bool two = b0 + 128 < row_bytes;
                tc::mbar_expect_tx(bar, two ? 4u * BOX_BYTES : 2u * BOX_BYTES);
                tc::tma_load_2d(st, &f.m->map, b0, row0, bar);
                tc::tma_load_2d(st + BOX_BYTES, &f.m->map, b0, row0 + f.second, bar);
                if (two) {
                    tc::tma_load_2d(st + 2 * BOX_BYTES, &f.m->map, b0 + 128, row0, bar);
                    tc::tma_load_2d(st + 3 * BOX_BYTES, &f.m->map, b0 + 128, row0 + f.second, bar);
                }
                s.next();
            }
        }
    }
}

// What a stage holds beside its weights: the rows' scale bytes, widened to
// 16-byte boundaries (every matrix of scales ends on one), and the pairs'
// activations.  A warp takes 0.35 us a stage for it, as long as HBM needs for the
// weights: a warp per stream keeps up.
template <int FMT>
__device__ __forceinline__ void stream_aux(const Params& p, const Shared& sh, uint32_t ring, int stream)
{
    using F = Format<FMT>;
    constexpr int PIECES = F::SCALE_PITCH / 16;              // of 16 bytes, per row
    const int lane = threadIdx.x & 31;
    const uint32_t aux0 = ring + (uint32_t)sh.plan.stages * WEIGHT_BYTES, aux_bytes = sh.plan.aux_bytes;
    const uint32_t act_at = sh.plan.acts_at + (uint32_t)(lane * F::RECORD), inverse_at = sh.plan.inverse_at + 4u * lane;
    Slots s(sh, stream);
    fence_async();                                           // x was converted by ordinary stores
    for (int which = 0; which < 2; ++which) {
        const Phase f = phase_of(p, sh.plan, which);
        const int srb = f.k / (FMT == kNv ? 16 : 32), stages = which == 0 ? p.xstages : p.hstages;
        bool ready = which == 0;
        for (Item it(f, stream); it.left > 0; it.next(f)) {
            const int g = it.group, tile = it.tile, n = sh.g_count[g];
            const int row0 = sh.g_expert[g] * f.rows + tile * f.step;
            // this lane's rows: lane of each box; where their bytes begin, rounded down, and by how much
            const uint8_t* src[2];
            int lead[2];
            if constexpr (FMT != kF8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t at = (int64_t)(row0 + i * f.second + lane) * srb;
                    src[i] = static_cast<const uint8_t*>(f.m->scales) + (at & ~(int64_t)15);
                    lead[i] = (int)(at & 15);
                    if (tile * f.step + i * f.second + lane >= f.rows) lead[i] = -(1 << 30);     // past the expert: nothing
                }
            }
            int row = 0;                                     // lane c: of pair c
            if (lane < n) {
                row = sh.list[sh.g_first[g] + lane];
                if (which == 0) row /= p.top_k;
            }
            const uint8_t* acts = (which == 0 ? p.xs : p.h) + (int64_t)row * stages * F::RECORD;
            float pow, inv = 0.0f;
            if (ready && which == 1 && lane < n) power_of(__ldcg(p.hmax + row), pow, inv);
            for (int i = 0; i < stages; ++i) {
                const bool ok = s.wait_empty(p.fault);
                if (!__all_sync(0xffffffffu, ok)) return;
                const uint32_t aux = aux0 + (uint32_t)s.at * aux_bytes, bar = s.full0 + 8u * s.at;
                if constexpr (FMT != kF8) {
                    const int from = i * F::SCALE_BYTES, want = min(F::SCALE_BYTES, srb - from);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint8_t* a = src[j] + from;
                        const uint32_t to = aux + (uint32_t)((32 * j + lane) * F::SCALE_PITCH);
#pragma unroll
                        for (int piece = 0; piece < PIECES; ++piece)
                            if (16 * piece < want + lead[j]) cp_async16(to + 16u * piece, a + 16 * piece, 16u);
                    }
                }
                if (!ready) {                                // down items: once all of h is written
                    const bool all = lane != 0 || spin(&p.ctl->h_done, gridDim.x, p.fault);
                    if (!__all_sync(0xffffffffu, all)) return;
                    fence_async();
                    if (lane < n) power_of(__ldcg(p.hmax + row), pow, inv);
                    ready = true;
                }
                if (which == 1 && lane < n)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(aux + inverse_at), "f"(inv) : "memory");
                // one arrival per lane, when its copies have landed; one for the inverses and the records' bytes
                if constexpr (FMT != kF8)
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
                __syncwarp();
                if (lane == 0) tc::mbar_expect_tx(bar, (uint32_t)(n * F::RECORD));
                __syncwarp();
                if (lane < n) tc::bulk_load(aux + act_at, acts + i * F::RECORD, (uint32_t)F::RECORD, bar);
                s.next();
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

// The same onto zeros.
__device__ __forceinline__ void mma16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four E8M0 scales as fp32 patterns' upper halves, two a word, in order: 2^(byte - 127), byte 255 NaN.
__device__ __forceinline__ void e8m0_four(uint32_t four, uint32_t (&two)[2])
{
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
        : "=r"(two[0]), "=r"(two[1])
        : "r"(four));
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

// Two UE4M3 bytes as f16; the conversion takes a byte's top bit for a sign (see the end of item).
__device__ __forceinline__ uint32_t ue4m3_pair(uint32_t c)
{
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(c));
    return h;
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
__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ void sums_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * STREAMS * SUM_WARPS) : "memory"); }

template <int N>
struct Int {
    static constexpr int value = N;
};

// A place in a stream's sequence of stages.
struct Cursor {
    uint32_t full0, empty0;
    int stages, slot;
    uint32_t phase, seq;            // of its stages so far
    bool live;
};

// One item's products: this warp's slice of k and half of the rows, acc[box][tile
// of 8 columns].  MMA row g stands for row (g / 2) + 4 (g % 2) of 8: with the
// 128-byte swizzle, two neighbouring g then read different halves of a row's
// 128 bytes, and a 16-byte read by all lanes hits every bank.  The order of k
// inside a product is free as long as both operands share it (see place).
template <int FMT, int NT, int WHICH>
__device__ __forceinline__ void item(const Params& p, const Plan& q, uint32_t ring, const Phase& f, int row0, int n,
                                     Cursor& cur, float (&acc)[2][NT][4])
{
    using F = Format<FMT>;
    const uint32_t full0 = cur.full0, empty0 = cur.empty0, aux0 = ring + (uint32_t)cur.stages * WEIGHT_BYTES;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3, half = (warp >> 2) & 1;
    const int rho = (g >> 1) | ((g & 1) << 2);
    const int srb = FMT == kNv ? f.k / 16 : f.k / 32;
    const float* f8_scales = nullptr;                        // of this item's first box
    int f8_second = 0;
    if (FMT == kF8) {
        f8_scales = static_cast<const float*>(f.m->scales) + (int64_t)(row0 >> 7) * (f.k >> 7);
        f8_second = ((row0 + f.second) >> 7) * (f.k >> 7) - (row0 >> 7) * (f.k >> 7);
    }
    // where the scale bytes of this lane's rows lie: a stage's copies begin at a multiple of 16 bytes of each row's
    // place in memory, so what precedes the bytes asked for is the same all through the item
    uint32_t scale_at[2][2] = {};
    if constexpr (FMT != kF8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t row = (uint32_t)(16 * half + 8 * r + rho);
                scale_at[i][r] = (32u * i + row) * F::SCALE_PITCH + (((uint32_t)(row0 + i * f.second) + row) * (uint32_t)srb & 15u);
            }
    }
    uint32_t seen[2][2] = {};                                // NVFP4: the scale bytes of this lane's rows, or'ed
    int col[NT];                                             // columns past the last pair repeat it
#pragma unroll
    for (int c = 0; c < NT; ++c) col[c] = min(8 * c + g, n - 1);

    for (int k0 = 0; k0 < f.k; k0 += F::VALUES) {
        const int s = cur.slot;
        const uint32_t ph = cur.phase;
        if ((cur.slot += STREAMS) >= cur.stages) cur.slot -= cur.stages, cur.phase ^= 1u;
        // turns, also from one item to the next, so that short stages load all warps alike (whose partial sums these are: item_products)
        const int qi = (int)(((uint32_t)warp + cur.seq++) & 3u);
        const int values = min(F::VALUES, f.k - k0);
        float fs[2] = {};
        if (FMT == kF8 && qi * F::QUARTER < values) {
#pragma unroll
            for (int i = 0; i < 2; ++i) fs[i] = __ldg(f8_scales + i * f8_second + (k0 >> 7) + (qi >> 1));
        }
        if (cur.live) cur.live = __all_sync(0xffffffffu, tc::wait_phase(full0 + 8u * s, ph, p.fault));
        if (qi * F::QUARTER < values) {
            const uint32_t aux = aux0 + (uint32_t)s * q.aux_bytes;
            const uint32_t w0 = ring + (uint32_t)(s * WEIGHT_BYTES + (qi >> 1) * 2 * BOX_BYTES + (16 * half + rho) * 128);
            const int c16 = 4 * (qi & 1);                    // of the row's 16-byte chunks, this quarter's first
            const int left = (values - qi * F::QUARTER + 31) / 32;     // blocks of 32 in this quarter, at least
            uint32_t act[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c)
                act[c] = aux + q.acts_at + (uint32_t)(col[c] * F::RECORD + qi * F::QUARTER * 2 + 16 * t);

            if constexpr (FMT == kMx) {
                // four blocks of 32; a lane holds values 8 t .. 8 t + 7 of each
                uint32_t sc[2][2][2];                        // two scales a word
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t at = aux + scale_at[i][r] + 4u * qi;
                        // four bytes that may straddle two words (one block may follow the last: not used)
                        const uint32_t lo = lds32(at & ~3u), hi = lds32((at & ~3u) + 4u * ((at & 3u) != 0u));
                        e8m0_four(__funnelshift_r(lo, hi, 8u * (at & 3u)), sc[i][r]);
                    }
                f32x2 ratio[NT][2];
                if constexpr (WHICH == 1) {
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const uint32_t pa = aux + q.acts_at + (uint32_t)(col[c] * F::RECORD + F::POWERS);
                        const float inv = as_f32(lds32(aux + q.inverse_at + 4u * col[c]));
                        lds_pairs(pa + 16u * qi, ratio[c][0], ratio[c][1]);
                        ratio[c][0] = mul2(ratio[c][0], pk(inv, inv));
                        ratio[c][1] = mul2(ratio[c][1], pk(inv, inv));
                    }
                }
                // block by block: with all blocks' loads ahead of the products it took 10 % longer (registers)
                const uint32_t wq = w0 + ((uint32_t)(c16 ^ (rho & 4)) << 4) + 4u * t;
                auto block = [&](auto which_block) {
                    constexpr int b = decltype(which_block)::value;
                    uint4 bf[NT];
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        bf[c] = lds128(act[c] + 64u * b);
                        if constexpr (WHICH == 1) {
                            float r0, r1;
                            upk(ratio[c][b >> 1], r0, r1);
                            const uint32_t m = (b & 1) ? f16x2(r1, r1) : f16x2(r0, r0);
                            bf[c].x = mul_f16x2(bf[c].x, m), bf[c].y = mul_f16x2(bf[c].y, m);
                            bf[c].z = mul_f16x2(bf[c].z, m), bf[c].w = mul_f16x2(bf[c].w, m);
                        }
                    }
                    const uint32_t wb = wq + ((uint32_t)(b ^ (rho & 3)) << 4);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t a0[4], a1[4];
                        widen4(lds32(wb + (uint32_t)(i * BOX_BYTES)), a0);
                        widen4(lds32(wb + (uint32_t)(i * BOX_BYTES + 1024)), a1);
                        const uint32_t p0 = sc[i][0][b >> 1], p1 = sc[i][1][b >> 1];
                        const float s0 = b & 1 ? bf16_hi(p0) : bf16_lo(p0), s1 = b & 1 ? bf16_hi(p1) : bf16_lo(p1);
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            float d[4];
                            mma16_zero(d, a0[0], a1[0], a0[1], a1[1], bf[c].x, bf[c].y);
                            mma16(d, a0[2], a1[2], a0[3], a1[3], bf[c].z, bf[c].w);
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[i][c][j] = __fmaf_rn(d[j], j < 2 ? s0 : s1, acc[i][c][j]);
                        }
                    }
                };
                block(Int<0>{});
                if (left > 1) block(Int<1>{});
                if (left > 2) block(Int<2>{});
                if (left > 3) block(Int<3>{});
            } else {
                constexpr int PIECES = FMT == kNv ? 4 : 2;   // 16-byte pieces of activations per lane
                uint4 bf[NT][PIECES], w[2][2];               // all loads first
                const uint32_t wa = w0 + ((uint32_t)((c16 + t) ^ rho) << 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (NT > 1 && i > 0) break;              // (of one box at a time with two tiles of columns: registers)
                    w[i][0] = lds128(wa + (uint32_t)(i * BOX_BYTES));
                    w[i][1] = lds128(wa + (uint32_t)(i * BOX_BYTES + 1024));
                }
                uint32_t two[2][2];                          // NVFP4: two scale bytes per row and block
                if constexpr (FMT == kNv) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            two[i][r] = t < left ? lds16(aux + scale_at[i][r] + 2u * (4 * qi + t)) : 0u;   // past the row: zeros
                            seen[i][r] |= two[i][r];
                        }
                }
#pragma unroll
                for (int c = 0; c < NT; ++c) {
#pragma unroll
                    for (int j = 0; j < PIECES; ++j) bf[c][j] = lds128(act[c] + 64u * j);
                    if constexpr (WHICH == 1) {
                        const uint32_t pa = aux + q.acts_at + (uint32_t)(col[c] * F::RECORD + F::POWERS);
                        const int block = FMT == kNv ? 4 * qi + t : 2 * qi + (t >> 1);
                        const float r = __fmul_rn(as_f32(lds32(pa + 4u * block)), as_f32(lds32(aux + q.inverse_at + 4u * col[c])));
                        const uint32_t m = f16x2(r, r);
#pragma unroll
                        for (int j = 0; j < PIECES; ++j) {
                            bf[c][j].x = mul_f16x2(bf[c][j].x, m), bf[c][j].y = mul_f16x2(bf[c][j].y, m);
                            bf[c][j].z = mul_f16x2(bf[c][j].z, m), bf[c][j].w = mul_f16x2(bf[c][j].w, m);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v0 = w[NT > 1 ? 0 : i][0], v1 = w[NT > 1 ? 0 : i][1];
                    const uint32_t u0[4] = {v0.x, v0.y, v0.z, v0.w}, u1[4] = {v1.x, v1.y, v1.z, v1.w};
                    if constexpr (FMT == kNv) {
                        uint32_t m[2][2];                    // two scales per row and block
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t h = ue4m3_pair(two[i][r]);
                            m[r][0] = __byte_perm(h, h, 0x1010);
                            m[r][1] = __byte_perm(h, h, 0x3232);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t a0[4], a1[4];
                            widen4(u0[j], a0);
                            widen4(u1[j], a1);
#pragma unroll
                            for (int l = 0; l < 4; ++l) {
                                a0[l] = mul_f16x2(a0[l], m[0][j >> 1]);
                                a1[l] = mul_f16x2(a1[l], m[1][j >> 1]);
                            }
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                mma16(acc[i][c], a0[0], a1[0], a0[1], a1[1], bf[c][j].x, bf[c][j].y);
                                mma16(acc[i][c], a0[2], a1[2], a0[3], a1[3], bf[c][j].z, bf[c][j].w);
                            }
                        }
                    } else {
                        float d[NT][4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t a0[4], a1[4];
                            widen8(u0[2 * j], u0[2 * j + 1], a0);
                            widen8(u1[2 * j], u1[2 * j + 1], a1);
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                if (j == 0)
                                    mma16_zero(d[c], a0[0], a1[0], a0[1], a1[1], bf[c][j].x, bf[c][j].y);
                                else
                                    mma16(d[c], a0[0], a1[0], a0[1], a1[1], bf[c][j].x, bf[c][j].y);
                                mma16(d[c], a0[2], a1[2], a0[3], a1[3], bf[c][j].z, bf[c][j].w);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < NT; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[i][c][j] = __fmaf_rn(d[c][j], fs[i], acc[i][c][j]);
                    }
                    if (NT > 1 && i == 0) {
                        w[0][0] = lds128(wa + BOX_BYTES);
                        w[0][1] = lds128(wa + BOX_BYTES + 1024u);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty0 + 8u * s);
    }
    if constexpr (FMT == kNv) {
        // A byte from 0x80 on is NaN (ue4m3_decode), and was taken for a negative scale: its row's sums become NaN
        // here, once an item (64 tokens over the wide layer 314 us; each byte turned into NaN on its way, 316).
        uint32_t flags = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) flags |= (seen[i][r] & 0x8080u) ? 1u << (2 * i + r) : 0u;
        if (__any_sync(0xffffffffu, flags != 0u)) {
            flags |= __shfl_xor_sync(0xffffffffu, flags, 1);             // the four lanes that share rows
            flags |= __shfl_xor_sync(0xffffffffu, flags, 2);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (flags >> (2 * i + (j >> 1)) & 1u) acc[i][c][j] = as_f32(0x7fc00000u);
        }
    }
}

// A place in a stream's sequence of buffers of partial sums.
struct Buffers {
    uint32_t summed, summable;      // the stream's barriers
    float* sums;                    // and its shared memory
    int n, at;
    uint32_t phase;
    __device__ __forceinline__ void next()
    {
        if (++at == n) at = 0, phase ^= 1u;
    }
};

// The product warps' part of one phase.
template <int FMT, int NT, int WHICH>
__device__ __forceinline__ void item_products(const Params& p, const Shared& sh, uint32_t ring, const Phase& f, int row0,
                                              int n, Cursor& cur, Buffers& buf)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // The slice is the quarter that the warp takes of the item's first stage: what a slice holds, and so the order
    // of the sums, does not depend on how many stages the stream has been through.
    const int slice = (int)(((uint32_t)warp + cur.seq) & 3u);
    float acc[2][NT][4] = {};
    item<FMT, NT, WHICH>(p, sh.plan, ring, f, row0, n, cur, acc);

    const int g = lane >> 2, t = lane & 3, half = (warp >> 2) & 1;
    constexpr int PITCH = 8 * NT + 1;                        // floats per row of the partial sums
    const int rho = (g >> 1) | ((g & 1) << 2);
    if (cur.live) cur.live = __all_sync(0xffffffffu, tc::wait_phase(buf.summed + 8u * buf.at, buf.phase ^ 1u, p.fault));
    float* to = buf.sums + (buf.at * SLICES * TILE + slice * TILE + 16 * half + rho) * PITCH + 2 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) to[(32 * i + 8 * (j >> 1)) * PITCH + 8 * c + (j & 1)] = acc[i][c][j];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(buf.summable + 8u * buf.at);
    buf.next();
}

template <int FMT, int WHICH>
__device__ __forceinline__ void multiply(const Params& p, const Shared& sh, uint32_t ring, int stream, Cursor& cur, Buffers& buf)
{
    const Phase f = phase_of(p, sh.plan, WHICH);
    for (Item it(f, stream); it.left > 0; it.next(f)) {
        const int n = sh.g_count[it.group], row0 = sh.g_expert[it.group] * f.rows + it.tile * f.step;
        if (n > 8)
            item_products<FMT, 2, WHICH>(p, sh, ring, f, row0, n, cur, buf);
        else
            item_products<FMT, 1, WHICH>(p, sh, ring, f, row0, n, cur, buf);
    }
}

// The summing warps' part: the four slices of k, in order, to h (WHICH 0) or
// to the pairs' results (1), beside the next item's products.
template <int FMT, int WHICH>
__device__ __forceinline__ void add_slices(const Params& p, const Shared& sh, int stream, Buffers& buf, bool& live)
{
    using F = Format<FMT>;
    const Phase f = phase_of(p, sh.plan, WHICH);
    const int lane = threadIdx.x & 31, warp = ((threadIdx.x >> 5) - FIRST_SUM) % SUM_WARPS;
    for (Item it(f, stream); it.left > 0; it.next(f), buf.next()) {
        const int grp = it.group, tile = it.tile, e = sh.g_expert[grp], n = sh.g_count[grp];
        const uint16_t* list = sh.list + sh.g_first[grp];
        const float gs = FMT == kNv && f.m->gscale ? __ldg(f.m->gscale + e * f.m->gstride) : 1.0f;
        float pow = 0.0f, inv;                               // lane c: of column c
        if (lane < n) {
            if (WHICH == 0)
                pow = __ldcg(p.xpow + list[lane] / p.top_k);
            else
                power_of(__ldcg(p.hmax + list[lane]), pow, inv);
        }
        if (live) live = __all_sync(0xffffffffu, tc::wait_phase(buf.summable + 8u * buf.at, buf.phase, p.fault));
        const int pitch = n > 8 ? 17 : 9;
        const float* from = buf.sums + (buf.at * SLICES * TILE + lane) * pitch;
        // a warp per pair, a lane for rows l and l + 32
        for (int c = warp; c < n; c += SUM_WARPS) {
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int k = 0; k < SLICES; ++k) {
                a += from[k * TILE * pitch + c];
                b += from[(k * TILE + 32) * pitch + c];
            }
            const float pw = __shfl_sync(0xffffffffu, pow, c);
            a = __fmul_rn(__fmul_rn(a, gs), pw);
            b = __fmul_rn(__fmul_rn(b, gs), pw);
            const int64_t pair = list[c];
            if (WHICH == 0) {
                // 32 consecutive values of h share a power of two
                const float v = __fmul_rn(__fdiv_rn(a, 1.0f + expf(-a)), b);
                const uint32_t top = __reduce_max_sync(0xffffffffu, finite_bits(v));
                float own;
                power_of(top, own, inv);
                uint8_t* rec = p.h + (pair * p.hstages + tile / F::BLOCKS) * F::RECORD;
                const int block = tile % F::BLOCKS;
                *reinterpret_cast<__half*>(rec + 2 * place<FMT>(block * 32 + lane)) = __float2half_rn(__fmul_rn(v, inv));
                if (lane == 0) {
                    *reinterpret_cast<float*>(rec + F::POWERS + 4 * block) = own;
                    atomicMax(p.hmax + pair, top);
                }
                if (tile == f.tiles - 1)                     // zeros to the end of the last record
                    for (int k = block + 1; k < F::BLOCKS; ++k) {
                        *reinterpret_cast<__half*>(rec + 2 * place<FMT>(k * 32 + lane)) = __float2half_rn(0.0f);
                        if (lane == 0) *reinterpret_cast<float*>(rec + F::POWERS + 4 * k) = 0.0f;
                    }
            } else {
                float* o = p.o + pair * p.hidden + tile * TILE + lane;
                o[0] = a;
                if (tile * TILE + 32 < p.hidden) o[32] = b;
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(buf.summed + 8u * buf.at);
    }
}

// One more CTA at a counter; what it held before.  A counter that was not zero before the call lets waits pass too
// early: one of the CTAs then finds it at `limit` (all CTAs) or above, and the fault word tells the caller.
__device__ __forceinline__ unsigned int count(unsigned int* counter, unsigned int limit, unsigned int* fault)
{
    const unsigned int before = atomicAdd(counter, 1u);
    if (before >= limit) atomicExch(fault, 1u);
    return before;
}

// All of this CTA's summing warps have stored: count it.
__device__ __forceinline__ void sums_count(const Params& p, unsigned int* counter)
{
    sums_sync();
    if (threadIdx.x == 32 * FIRST_SUM) {
        __threadfence();
        count(counter, gridDim.x, p.fault);
    }
}

// All threads of all CTAs, for the n-th time.
__device__ __forceinline__ void all_ctas(const Params& p, unsigned int n)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        count(&p.ctl->start, n * gridDim.x, p.fault);
        spin(&p.ctl->start, n * gridDim.x, p.fault);
    }
    __syncthreads();
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
            // the weights' bytes; the lanes that copy scale bytes; the records' bytes
            tc::mbar_init(smem_of(&sh.full[i]), 1u + (FMT == kF8 ? 0u : 32u) + 1u);
            tc::mbar_init(smem_of(&sh.empty[i]), (uint32_t)SET);
        }
        for (int i = 0; i < 2 * STREAMS; ++i) {
            tc::mbar_init(smem_of(&sh.summable[i / 2][i % 2]), (uint32_t)SET);
            tc::mbar_init(smem_of(&sh.summed[i / 2][i % 2]), (uint32_t)SUM_WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.up.map)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.down.map)) : "memory");
    }
    convert_x<FMT>(p, reinterpret_cast<unsigned int*>(red));
    if (p.router) route_logits(p);
    all_ctas(p, 1u);
    // A few tokens every CTA chooses for by itself.  More are shared out, a CTA a
    // token: another wait for all CTAs, 1.3 us, but every CTA reading all logits
    // took 15 us for 64 tokens of 64 experts.
    const bool shared_out = p.router && p.tokens > 8;
    if (p.router && (!shared_out || warp == 0)) {
        const int first = shared_out ? (int)blockIdx.x : warp, step = shared_out ? (int)gridDim.x : THREADS / 32;
        const bool tell = shared_out || blockIdx.x == 0;
        if (p.experts <= 32)
            choose<1>(p, sh, first, step, tell);
        else if (p.experts <= 128)
            choose<4>(p, sh, first, step, tell);
        else
            choose<MAX_EXPERTS / 32>(p, sh, first, step, tell);
    }
    if (shared_out) all_ctas(p, 2u);
    if (shared_out || !p.router) {
        for (int i = threadIdx.x; i < p.tokens * p.top_k; i += THREADS) {
            const int e = __ldcg(p.ids + i);
            sh.id[i] = (unsigned)e < (unsigned)p.experts ? (uint16_t)e : (uint16_t)NONE;
            sh.w[i] = __ldcg(p.weights + i);
        }
    }
    __syncthreads();
    make_plan<FMT>(p, sh);

    const int stream = warp < FIRST_COPY ? warp / SET : warp < FIRST_SUM ? (warp - FIRST_COPY) / 2 : (warp - FIRST_SUM) / SUM_WARPS;
    Buffers buf{smem_of(sh.summed[stream]), smem_of(sh.summable[stream]), red + stream * (RED_BYTES / 4 / STREAMS),
                sh.plan.buffers, 0, 0u};
    if (warp < FIRST_COPY) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_PRODUCTS));
        Cursor cur{smem_of(sh.full), smem_of(sh.empty), sh.plan.stages, stream, 0u, 0u, true};
        multiply<FMT, 0>(p, sh, ring, stream, cur, buf);
        multiply<FMT, 1>(p, sh, ring, stream, cur, buf);
    } else if (warp < FIRST_SUM) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHERS));
        if (warp & 1) {
            stream_aux<FMT>(p, sh, ring, stream);
        } else {
            if ((threadIdx.x & 31) == 0) stream_weights<FMT>(p, sh, ring, stream);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHERS));
        bool live = true;
        add_slices<FMT, 0>(p, sh, stream, buf, live);
        sums_count(p, &p.ctl->h_done);
        // the pairs' maxima are read directly, not through a stage
        if (threadIdx.x == 32 * FIRST_SUM) spin(&p.ctl->h_done, gridDim.x, p.fault);
        sums_sync();
        add_slices<FMT, 1>(p, sh, stream, buf, live);
        sums_count(p, &p.ctl->o_done);
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
            if (sh.id[pair] == NONE) continue;
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
        if (count(&p.ctl->leaving, gridDim.x, p.fault) == gridDim.x - 1) {
            p.ctl->start = p.ctl->h_done = p.ctl->o_done = 0u;
            __threadfence();
            p.ctl->leaving = 0u;
        }
    }
}

// ---------------------------------------------------------------- host
// Stages and bytes of a row of records (Format::VALUES, RECORD).
int64_t stages_of(int64_t values, int fmt) { return fmt == kF8 ? (values + 255) / 256 : (values + 511) / 512; }
int64_t record_bytes(int fmt) { return fmt == kF8 ? Format<kF8>::RECORD : Format<kNv>::RECORD; }
static_assert(Format<kF8>::VALUES == 256 && Format<kNv>::VALUES == 512 && Format<kMx>::VALUES == 512 &&
                  Format<kMx>::RECORD == Format<kNv>::RECORD,
              "stages_of and record_bytes");

struct Layout {
    size_t logits, xs, xpow, h, hmax, o, total;
};

Layout layout(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k, int fmt)
{
    auto up = [](int64_t v) { return (size_t)((v + 255) & ~(int64_t)255); };
    const int64_t pairs = tokens * top_k, rec = record_bytes(fmt);
    Layout l;
    l.logits = 256;
    l.xs = l.logits + up(8 * tokens * experts * 8);
    l.xpow = l.xs + up(tokens * stages_of(hidden, fmt) * rec);
    l.h = l.xpow + up(tokens * 4);
    l.hmax = l.h + up(pairs * stages_of(inter, fmt) * rec);
    l.o = l.hmax + up(pairs * 4);
    l.total = l.o + up(pairs * hidden * 4);
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
    // a record per 512 FP4 values or two per 512 E4M3 values: room for either
    const size_t a = fp4q::moe::layout(tokens, hidden, inter, experts, top_k, fp4q::moe::kF8).total;
    const size_t b = fp4q::moe::layout(tokens, hidden, inter, experts, top_k, fp4q::moe::kNv).total;
    return a > b ? a : b;
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
    const Layout l = layout(tokens, hidden, inter, experts, top_k, fmt);
    if (ws_bytes < fp4q_moe_workspace_size(tokens, hidden, inter, experts, top_k)) return FP4Q_ERR_WORKSPACE;

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
    p.logits = reinterpret_cast<double*>(ws + l.logits);
    p.xs = reinterpret_cast<uint8_t*>(ws + l.xs);
    p.xpow = reinterpret_cast<float*>(ws + l.xpow);
    p.h = reinterpret_cast<uint8_t*>(ws + l.h);
    p.hmax = reinterpret_cast<unsigned int*>(ws + l.hmax);
    p.o = reinterpret_cast<float*>(ws + l.o);
    p.tokens = (int)tokens;
    p.hidden = (int)hidden;
    p.inter = (int)inter;
    p.experts = (int)experts;
    p.top_k = (int)top_k;
    p.normalize = normalize != 0;
    p.xstages = (int)stages_of(hidden, fmt);
    p.hstages = (int)stages_of(inter, fmt);
    p.fault = device_fault_word();
    if (!p.fault) return FP4Q_ERR_CUDA;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (fmt == kMx) return launch<kMx>(p, cs);
    if (fmt == kNv) return launch<kNv>(p, cs);
    return launch<kF8>(p, cs);
}


// fp4q_f8_gemm.cu -- matrix product of two E4M3 operands with one fp32 scale
// for each block of 128 along k:
//   y[i][j] = sum_b sA[i][b] sB[j / 128][b] sum_{k in block b} a[i][k] b[j][k].
//
// The tensor cores take no fp32 scale, so the sum over one block of 128 is
// formed in tensor memory (tcgen05.mma kind::f8f6f4, four instructions of
// K = 32) and added, scaled, to running fp32 sums in registers:
//   acc = fma(partial, fp32(sA sB), acc).
//
// A persistent grid (one CTA per SM) walks the 128 x BN tiles of y; each tile
// walks k in blocks of 128 bytes through a ring of shared-memory stages:
//   warp 0, one thread: TMA loads of the A and B code tiles;
//   warps 1 and 2 (warp 1 also allocates tensor memory): one thread each issues
//     every other block's MMAs into the next of 512 / BN accumulators, so block
//     b + 1 runs while block b is drained.  One thread alone took 650 clocks a
//     block for its two waits and two commits, more than the 512 of the MMAs;
//   warps 4-11: two groups of four, each draining half the columns: a thread
//     owns a row of y (a lane of tensor memory) and BN / 2 columns, and the scale
//     is one number per thread and block.
// For few rows of A a second kernel (below) puts B's rows on the lanes instead.
// Every wait is bounded; a wait that runs out records the library's fault word
// and the CTA stops its work and returns.
//
// Measured, in a loop of calls: 8192 x 13824 x 5120 658 us under the power cap,
// 1.76 PFLOP/s (0.53 of twice the measured bf16 rate); in graph replays on a cool
// chip 566, of 351 at that rate, and 490 with the accumulators left unread: the
// operands' way from L2 costs 139 us over the floor, the sums' way out of tensor
// memory 76.  1 x 13824 x 5120 15.7 us (its bytes at the copy rate: 10.8); 37 x
// 3584 x 18944 17.9 (10.5).
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstring>

#include "fp4q_device.cuh"
#include "fp4q_launch.h"
#include "fp4q_tc.cuh"
#include "fp4q_tma.h"
#include "../../include/fp4q.h"

namespace fp4q {
namespace f8gemm {

constexpr int BM = 128, BK = 128;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (4 + EPI_WARPS);       // three warpgroups: control, two epilogue groups
constexpr int REGS_CONTROL = 40, REGS_EPI = 232;    // 128 x 40 + 256 x 232 = 384 x 168, the launch's registers
constexpr int ISSUERS = 2;                          // warps that issue MMAs, a block of k in turn
constexpr uint32_t TMEM_COLS = 512;

template <int BN>
struct Shape {
    static constexpr int A_BYTES = BM * BK;
    static constexpr int STAGE_BYTES = A_BYTES + BN * BK;
    static constexpr int NSTAGE = ((192 * 1024) / STAGE_BYTES) & ~1;
    static constexpr int NBUF = (int)TMEM_COLS / BN;
    static constexpr int SMEM_BYTES = 1024 + NSTAGE * STAGE_BYTES + 256 + EPI_WARPS * 32 * 33 * 4;
    static constexpr int HALF = BN / 2;                     // columns per epilogue group
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(16 * (NSTAGE + NBUF) + 8 <= 256, "barriers");
    // a slot of either ring belongs to one issuer: a barrier's parity tells only neighbouring phases apart
    static_assert(NSTAGE % ISSUERS == 0 && NBUF % ISSUERS == 0, "rings");
};

struct Params {
    CUtensorMap ta;                 // A codes [m][k] bytes, box 128 x 128
    CUtensorMap tb;                 // B codes [n][k] bytes, box BN x 128
    const float* sa;                // [m][kb]
    const float* sb;                // [ceil(n / 128)][kb]
    void* y;                        // [m][n]
    int64_t m, n, kb;
    int f32;
    unsigned int* fault;
};

// Instruction descriptor: D fp32 (bits 4-5 = 1), A and B E4M3 (bits 7-9 and
// 10-12 = 0), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__device__ __forceinline__ constexpr uint32_t idesc(int m, int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// tcgen05.ld without its wait, and the wait, which hands the registers on: what
// uses them cannot be moved before it.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// acc += s * v, 32 columns.  Scalar fused multiply-adds: as packed pairs the
// same sums took a quarter longer (8192 x 13824 x 5120: 781 against 618 us).
__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], float s)
{
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = __fmaf_rn(as_f32(v[j]), s, acc[j]);
}

// A warp's results: a thread has row r, HALF columns from c0.  Rows that 32-byte
// stores fit (n a multiple of 16, or of 8 for fp32) go out as they are, a sector
// a lane; others by way of the warp's corner of shared memory, 32 columns at a
// time, so that the lanes store neighbouring columns of one row.
template <int HALF>
__device__ __forceinline__ void store_rows(const Params& p, int64_t r, int64_t c0, const float (&acc)[HALF], float* corner)
{
    if (c0 >= p.n) return;
    const int64_t at = r * p.n + c0;
    const bool whole = c0 + HALF <= p.n;
    if (p.f32 && whole && (p.n & 7) == 0 && (reinterpret_cast<uintptr_t>(p.y) & 31u) == 0) {
        if (r >= p.m) return;
        float* dst = static_cast<float*>(p.y) + at;
#pragma unroll
        for (int j = 0; j < HALF; j += 8)
            stg256(dst + j, as_u32(acc[j]), as_u32(acc[j + 1]), as_u32(acc[j + 2]), as_u32(acc[j + 3]), as_u32(acc[j + 4]),
                   as_u32(acc[j + 5]), as_u32(acc[j + 6]), as_u32(acc[j + 7]));
    } else if (!p.f32 && whole && (p.n & 15) == 0 && (reinterpret_cast<uintptr_t>(p.y) & 31u) == 0) {
        if (r >= p.m) return;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.y) + at;
#pragma unroll
        for (int j = 0; j < HALF; j += 16) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = bf16x2(acc[j + 2 * i], acc[j + 2 * i + 1]);
            stg256(dst + j, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
        }
    } else {
        const int lane = threadIdx.x & 31;
        const int64_t r0 = r - lane;
#pragma unroll
        for (int j = 0; j < HALF; j += 32) {
            if (c0 + j >= p.n) break;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i) corner[lane * 33 + i] = acc[j + i];
            __syncwarp();
            const int64_t col = c0 + j + lane;
            const int rows = (int)(p.m - r0 < 32 ? p.m - r0 : 32);
            if (col < p.n)
#pragma unroll 4
                for (int i = 0; i < rows; ++i) {
                    const float v = corner[i * 33 + lane];
                    if (p.f32)
                        static_cast<float*>(p.y)[(r0 + i) * p.n + col] = v;
                    else
                        static_cast<__nv_bfloat16*>(p.y)[(r0 + i) * p.n + col] = __float2bfloat16_rn(v);
                }
        }
        __syncwarp();
    }
}

// An epilogue thread's part of a tile: row r, HALF columns from c0, over all
// blocks of k; `release` hands an accumulator back.  False once a wait ran out.
template <int BN, int NBUF, typename Release>
__device__ __forceinline__ bool drain_tile(const Params& p, uint32_t tmem, uint32_t afull0, int half, int64_t r, int64_t c0,
                                           int& b, uint32_t& bph, float* corner, Release release)
{
    constexpr int HALF = BN / 2;
    const int warp = threadIdx.x >> 5, q = warp & 3;
    const float* sa = p.sa + (r < p.m ? r : p.m - 1) * p.kb;
    const float* sb = p.sb + ((c0 < p.n ? c0 : p.n - 1) >> 7) * p.kb;
    float acc[HALF];
#pragma unroll
    for (int j = 0; j < HALF; ++j) acc[j] = 0.0f;
    float a1 = __ldg(sa), b1 = __ldg(sb);
    for (int kt = 0; kt < (int)p.kb; ++kt) {
        const float s = __fmul_rn(a1, b1);
        const int nx = kt + 1 < (int)p.kb ? kt + 1 : kt;
        a1 = __ldg(sa + nx);
        b1 = __ldg(sb + nx);
        const bool done = tc::wait_phase(afull0 + 8u * b, bph, p.fault);
        if (!__all_sync(0xffffffffu, done)) return false;
        tc::tc_fence_after();
        // the next 32 columns are on their way while these are added
        const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * BN + half * HALF);
        uint32_t v[2][32];
        tmem_ld32_issue(at, v[0]);
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c) {
            tmem_ld_wait(v[c & 1]);
            if (c + 1 < HALF / 32) {
                tmem_ld32_issue(at + 32u * (uint32_t)(c + 1), v[(c + 1) & 1]);
            } else {
                tc::tc_fence_before();
                __syncwarp();
                release(b);
            }
            add_scaled(acc + 32 * c, v[c & 1], s);
        }
        if (++b == NBUF) b = 0, bph ^= 1u;
    }
    store_rows<HALF>(p, r, c0, acc, corner);
    return true;
}

// The persistent kernel's t-th tile: bands of 16 rows of tiles, down a column of
// the band, then the next column, so that the CTAs at work share about 16 tiles
// of A and 10 of B.  Down whole columns of a tall A, every column of tiles reads
// A anew from memory: 32768 x 13824 x 5120 took 2540 us, in bands it takes 2230
// (bands of 8: 2255); 8192 x 13824 x 5120, whose A stays in L2, 579 and 574.
constexpr int BAND = 16;

__device__ __forceinline__ void tile_at(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn)
{
    const int64_t first = t / (BAND * tiles_n) * BAND, in_band = t - first * tiles_n;
    const int64_t rows = tiles_m - first < BAND ? tiles_m - first : BAND;
    tm = first + in_band % rows;
    tn = in_band / rows;
}

template <int BN>
__global__ void __launch_bounds__(THREADS, 1) f8_gemm_kernel(const __grid_constant__ Params p)
{
    using S = Shape<BN>;
    extern __shared__ __align__(1024) uint8_t smem_f8[];
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_f8);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t full0 = base + S::NSTAGE * S::STAGE_BYTES, empty0 = full0 + 8u * S::NSTAGE;
    const uint32_t afull0 = empty0 + 8u * S::NSTAGE, aempty0 = afull0 + 8u * S::NBUF;
    const uint32_t slot = aempty0 + 8u * S::NBUF;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int64_t tiles_m = (p.m + BM - 1) / BM;
    const int64_t tiles_n = (p.n + BN - 1) / BN, n_tiles = tiles_m * tiles_n;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::NSTAGE; ++i) {
            tc::mbar_init(full0 + 8u * i, 1u);
            tc::mbar_init(empty0 + 8u * i, 1u);
        }
        for (int i = 0; i < S::NBUF; ++i) {
            tc::mbar_init(afull0 + 8u * i, 1u);
            tc::mbar_init(aempty0 + 8u * i, (uint32_t)EPI_WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(slot, TMEM_COLS);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

    pdl_wait();                                              // what came before in the stream; the set-up above overlaps it
    pdl_release();
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CONTROL));
        if (warp == 0 && lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.ta)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tb)) : "memory");
            int s = 0;
            uint32_t ph = 1;                                     // a fresh barrier's previous phase counts as completed
            bool ok = true;
            for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
                int64_t tm, tn;
                tile_at(t, tiles_m, tiles_n, tm, tn);
                const int m0 = (int)(tm * BM), n0 = (int)(tn * BN);
                for (int kt = 0; kt < (int)p.kb; ++kt) {
                    if (!tc::wait_phase(empty0 + 8u * s, ph, p.fault)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = base + (uint32_t)(s * S::STAGE_BYTES), fb = full0 + 8u * s;
                    tc::mbar_expect_tx(fb, (uint32_t)S::STAGE_BYTES);
                    tc::tma_load_2d(st, &p.ta, kt * BK, m0, fb);
                    tc::tma_load_2d(st + S::A_BYTES, &p.tb, kt * BK, n0, fb);
                    if (++s == S::NSTAGE) s = 0, ph ^= 1u;
                }
            }
        } else if (warp < 1 + ISSUERS && lane == 0) {
            // blocks mine, mine + ISSUERS, ... of this CTA's sequence
            const int mine = warp - 1;
            int s = mine, b = mine;
            uint32_t ph = 0, bph = 1;
            int64_t blocks = 0;
            for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x) blocks += p.kb;
            for (int64_t i = mine; i < blocks; i += ISSUERS) {
                if (!tc::wait_phase(aempty0 + 8u * b, bph, p.fault) || !tc::wait_phase(full0 + 8u * s, ph, p.fault)) break;
                tc::tc_fence_after();
                const uint32_t st = base + (uint32_t)(s * S::STAGE_BYTES);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8(tmem + (uint32_t)(b * BN), tc::sw128_desc(st + 32u * kk),
                           tc::sw128_desc(st + S::A_BYTES + 32u * kk), idesc(BM, BN), kk > 0);
                tc::mma_commit(empty0 + 8u * s);
                tc::mma_commit(afull0 + 8u * b);
                if ((s += ISSUERS) >= S::NSTAGE) s -= S::NSTAGE, ph ^= 1u;
                if ((b += ISSUERS) >= S::NBUF) b -= S::NBUF, bph ^= 1u;
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        const int half = (warp - 4) >> 2;
        float* corner = reinterpret_cast<float*>(smem_f8 + (base - raw) + S::NSTAGE * S::STAGE_BYTES + 256) + (warp - 4) * 32 * 33;
        int b = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
            int64_t tm, tn;
            tile_at(t, tiles_m, tiles_n, tm, tn);
            ok = drain_tile<BN, S::NBUF>(p, tmem, afull0, half, tm * BM + 32 * (warp & 3) + lane,
                                         tn * BN + half * S::HALF, b, bph, corner, [&](int buf) {
                                             if (lane == 0) tc::mbar_arrive(aempty0 + 8u * buf);
                                         });
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int BN>
int launch(Params& p, const uint8_t* b, int64_t k, cudaStream_t s)
{
    if (!make_byte_map(&p.tb, b, p.n, k, BN)) return FP4Q_ERR_CUDA;
    const int64_t tiles = ((p.m + BM - 1) / BM) * ((p.n + BN - 1) / BN);
    const int grid = grid_for((const void*)f8_gemm_kernel<BN>, Shape<BN>::SMEM_BYTES, tiles, THREADS);
    return launch_pdl(f8_gemm_kernel<BN>, grid, THREADS, Shape<BN>::SMEM_BYTES, s, p) == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// ---------------------------------------------------------------- few tokens
// With few rows of A the product is bound by B's bytes (or, at a few hundred
// rows, there are too few 128 x 128 tiles for the SMs), so B's rows take the
// 128 lanes of the MMA, up to NTOK rows of A its columns, and k is split over
// the CTAs of a cluster.  A lane of tensor memory is then a row of B: the
// scales vary along the columns and come from shared memory, where the CTA has
// multiplied fp32(sA sB) for its blocks beforehand.  At the end CTA r of the
// cluster adds every CTA's sums of its share of the columns, in rank order,
// through distributed shared memory: no workspace, no atomics, and 32 lanes
// store 32 neighbouring columns of a row of y.
template <int NTOK>
struct Small {
    static constexpr int B_BYTES = 128 * BK;
    static constexpr int STAGE_BYTES = B_BYTES + NTOK * BK;
    static constexpr int NSTAGE = NTOK == 16 ? 5 : 4;
    static constexpr int NBUF = 4;
    static constexpr uint32_t COLS = NBUF * NTOK;           // 64, 128, 256: two CTAs share an SM's 512
    static constexpr int SCALE_BYTES = NTOK <= 32 ? 16384 : 12288;
    static constexpr int SCALE_PITCH = NTOK + 4;            // floats per block of k
    static constexpr int MAX_KB = SCALE_BYTES / 4 / SCALE_PITCH;            // blocks of k per CTA
    static constexpr int SMEM_BYTES = 1024 + NSTAGE * STAGE_BYTES + SCALE_BYTES + 256;
    static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
    static_assert(NSTAGE * STAGE_BYTES >= NTOK * 128 * 4, "the partial sums reuse the ring");
};
constexpr int SMALL_THREADS = 32 * 6;

struct SmallParams {
    CUtensorMap ta;                 // A codes, box NTOK x 128
    CUtensorMap tb;                 // B codes, box 128 x 128
    const float* sa;
    const float* sb;
    void* y;
    int64_t m, n, kb;
    int f32, split;                 // CTAs per cluster
    unsigned int* fault;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void store_one(const SmallParams& p, int64_t row, int64_t col, float v)
{
    if (p.f32)
        static_cast<float*>(p.y)[row * p.n + col] = v;
    else
        static_cast<__nv_bfloat16*>(p.y)[row * p.n + col] = __float2bfloat16_rn(v);
}

template <int NTOK>
__global__ void __launch_bounds__(SMALL_THREADS, 2) f8_gemm_small_kernel(const __grid_constant__ SmallParams p)
{
    using S = Small<NTOK>;
    extern __shared__ __align__(1024) uint8_t smem_f8[];
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_f8);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t scales = base + S::NSTAGE * S::STAGE_BYTES;
    const uint32_t full0 = scales + S::SCALE_BYTES, empty0 = full0 + 8u * S::NSTAGE;
    const uint32_t afull0 = empty0 + 8u * S::NSTAGE, aempty0 = afull0 + 8u * S::NBUF, slot = aempty0 + 8u * S::NBUF;
    float* sums = reinterpret_cast<float*>(smem_f8 + (base - raw));          // over the ring, once it is done with
    float* sc = reinterpret_cast<float*>(smem_f8 + (scales - raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // cluster c: 128 rows of B, NTOK rows of A; its CTA `rank`: blocks from k0 to k1
    const int rank = (int)(blockIdx.x % (unsigned)p.split);
    const int64_t tile = blockIdx.x / (unsigned)p.split, tiles_m = (p.m + NTOK - 1) / NTOK;
    const int64_t m0 = (tile % tiles_m) * NTOK, n0 = (tile / tiles_m) * 128;
    const int k0 = (int)(p.kb * rank / p.split), k1 = (int)(p.kb * (rank + 1) / p.split), nk = k1 - k0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::NSTAGE; ++i) {
            tc::mbar_init(full0 + 8u * i, 1u);
            tc::mbar_init(empty0 + 8u * i, 1u);
        }
        for (int i = 0; i < S::NBUF; ++i) {
            tc::mbar_init(afull0 + 8u * i, 1u);
            tc::mbar_init(aempty0 + 8u * i, 4u);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(slot, S::COLS);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

    pdl_wait();
    pdl_release();
    f32x2 acc[NTOK / 2];
    if (warp == 0 && lane == 0) {
        for (int i = 0, s = 0, ph = 1; i < nk; ++i) {
            if (!tc::wait_phase(empty0 + 8u * s, (uint32_t)ph, p.fault)) break;
            const uint32_t st = base + (uint32_t)(s * S::STAGE_BYTES), fb = full0 + 8u * s;
            tc::mbar_expect_tx(fb, (uint32_t)S::STAGE_BYTES);
            tc::tma_load_2d(st, &p.tb, (k0 + i) * BK, (int)n0, fb);
            tc::tma_load_2d(st + S::B_BYTES, &p.ta, (k0 + i) * BK, (int)m0, fb);
            if (++s == S::NSTAGE) s = 0, ph ^= 1;
        }
    } else if (warp == 1 && lane == 0) {
        for (int i = 0, s = 0, ph = 0, b = 0, bph = 1; i < nk; ++i) {
            if (!tc::wait_phase(aempty0 + 8u * b, (uint32_t)bph, p.fault) ||
                !tc::wait_phase(full0 + 8u * s, (uint32_t)ph, p.fault))
                break;
            tc::tc_fence_after();
            const uint32_t st = base + (uint32_t)(s * S::STAGE_BYTES);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f8(tmem + (uint32_t)(b * NTOK), tc::sw128_desc(st + 32u * kk),
                       tc::sw128_desc(st + S::B_BYTES + 32u * kk), idesc(128, NTOK), kk > 0);
            tc::mma_commit(empty0 + 8u * s);
            tc::mma_commit(afull0 + 8u * b);
            if (++s == S::NSTAGE) s = 0, ph ^= 1;
            if (++b == S::NBUF) b = 0, bph ^= 1;
        }
    } else if (warp >= 2) {
        const int q = warp & 3;
        const float* sb = p.sb + (n0 >> 7) * p.kb + k0;
        // 32 lanes a row of A, four rows at a time
        for (int b = lane; b < nk; b += 32) {
            const float v = __ldg(sb + b);
            const float* a = p.sa + (m0 + q) * p.kb + k0 + b;
#pragma unroll
            for (int t = 0; t < NTOK / 4; ++t)
                sc[b * S::SCALE_PITCH + 4 * t + q] = m0 + 4 * t + q < p.m ? __fmul_rn(__ldg(a + 4 * t * p.kb), v) : 0.0f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int j = 0; j < NTOK / 2; ++j) acc[j] = 0ull;
        bool live = true;
        for (int i = 0, b = 0, bph = 0; i < nk; ++i) {
            if (live) live = __all_sync(0xffffffffu, tc::wait_phase(afull0 + 8u * b, (uint32_t)bph, p.fault));
            tc::tc_fence_after();
            const uint32_t row = scales + (uint32_t)(i * S::SCALE_PITCH * 4);
            constexpr int W = NTOK < 32 ? 16 : 32;
#pragma unroll
            for (int c = 0; c < NTOK / W; ++c) {
                uint32_t v[32];
                const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * NTOK + W * c);
                if constexpr (W == 16)
                    tmem_ld16(at, v);
                else
                    tc::tmem_ld32(at, v);
                if (c == NTOK / W - 1) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(aempty0 + 8u * b);
                }
#pragma unroll
                for (int j = 0; j < W / 4; ++j) {
                    f32x2 s0, s1;
                    lds_pairs(row + (uint32_t)((W * c + 4 * j) * 4), s0, s1);
                    f32x2& a0 = acc[(W * c + 4 * j) / 2];
                    f32x2& a1 = acc[(W * c + 4 * j) / 2 + 1];
                    a0 = fma2(pk(as_f32(v[4 * j]), as_f32(v[4 * j + 1])), s0, a0);
                    a1 = fma2(pk(as_f32(v[4 * j + 2]), as_f32(v[4 * j + 3])), s1, a1);
                }
            }
            if (++b == S::NBUF) b = 0, bph ^= 1;
        }
        if (p.split == 1) {
            const int64_t col = n0 + 32 * q + lane;
            if (col < p.n)
#pragma unroll
                for (int j = 0; j < NTOK / 2; ++j) {
                    float a, b;
                    upk(acc[j], a, b);
                    if (m0 + 2 * j < p.m) store_one(p, m0 + 2 * j, col, a);
                    if (m0 + 2 * j + 1 < p.m) store_one(p, m0 + 2 * j + 1, col, b);
                }
        }
    }
    if (p.split > 1) {
        // columns that each CTA adds (a power of two, at least 2), kept [rank][column][row of B]: a warp's stores to
        // another CTA are then 128 consecutive bytes (rows of `share` columns, 16 bytes a lane, took 1 us more)
        const int share = NTOK / p.split, log_share = __ffs(share) - 1, r = 32 * (warp & 3) + lane;
        __syncwarp();
        __syncthreads();                                     // the ring has been read: the commits were waited for
        cluster_sync();
        if (warp >= 2) {
            const uint32_t mine = (uint32_t)__cvta_generic_to_shared(sums + rank * share * 128 + r);
#pragma unroll
            for (int j = 0; j < NTOK; ++j) {
                float a, b;
                upk(acc[j / 2], a, b);
                uint32_t dst = mine + 512u * (uint32_t)(j & (share - 1));
                asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(dst) : "r"(j >> log_share));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(j & 1 ? b : a) : "memory");
            }
        }
        cluster_sync();
        if (warp >= 2 && n0 + r < p.n) {
            const int64_t row0 = m0 + rank * share;
            for (int j = 0; j < share; j += 2) {
                float a[2] = {0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < p.split) {
                        a[0] += sums[(k * share + j) * 128 + r];
                        a[1] += sums[(k * share + j + 1) * 128 + r];
                    }
                if (row0 + j < p.m) store_one(p, row0 + j, n0 + r, a[0]);
                if (row0 + j + 1 < p.m) store_one(p, row0 + j + 1, n0 + r, a[1]);
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, S::COLS);
    }
}

// The few-token product in tiles of 128 x NTOK over clusters of `split` CTAs.
template <int NTOK>
int launch_small(const Params& g, const uint8_t* a, const uint8_t* b, int64_t k, int split, cudaStream_t s)
{
    SmallParams p;
    memset(&p, 0, sizeof(p));
    if (!make_byte_map(&p.ta, a, g.m, k, NTOK) || !make_byte_map(&p.tb, b, g.n, k, 128)) return FP4Q_ERR_CUDA;
    p.sa = g.sa;
    p.sb = g.sb;
    p.y = g.y;
    p.m = g.m;
    p.n = g.n;
    p.kb = g.kb;
    p.f32 = g.f32;
    p.split = split;
    p.fault = g.fault;
    resident_ctas((const void*)f8_gemm_small_kernel<NTOK>, Small<NTOK>::SMEM_BYTES, SMALL_THREADS);   // opts in to the shared memory
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((g.m + NTOK - 1) / NTOK) * ((g.n + 127) / 128) * split));
    cfg.blockDim = dim3((unsigned)SMALL_THREADS);
    cfg.dynamicSmemBytes = Small<NTOK>::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, f8_gemm_small_kernel<NTOK>, p) == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// CTAs per cluster for `tiles` tiles of kb blocks: the most (8 at most) that all
// fit at two CTAs per SM and have two blocks each; 0 if a CTA's scales would not fit.
int split_of(int64_t tiles, int64_t kb, int max_kb)
{
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * 148 && kb >= 4 * split) split *= 2;
    while (split < 8 && (kb + split - 1) / split > max_kb) split *= 2;
    return (kb + split - 1) / split <= max_kb ? split : 0;
}

}  // namespace f8gemm
}  // namespace fp4q

extern "C" int fp4q_f8_gemm(const uint8_t* codes_a, const float* scales_a, int64_t m, const uint8_t* codes_b,
                            const float* scales_b, int64_t n, int64_t k, int out_dtype, void* y, void* stream)
{
    using namespace fp4q;
    if (m < 0 || n < 0 || k < 0 || k % 16 != 0) return FP4Q_ERR_SHAPE;
    if (m > INT32_MAX - 256 || n > INT32_MAX - 256 || k > INT32_MAX - 256) return FP4Q_ERR_SHAPE;   // tile coordinates are 32 bits
    if (out_dtype != FP4Q_OUT_BF16 && out_dtype != FP4Q_OUT_F32) return FP4Q_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return FP4Q_OK;
    if (!y) return FP4Q_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(y) & (out_dtype == FP4Q_OUT_F32 ? 3u : 1u)) return FP4Q_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k == 0)
        return cudaMemsetAsync(y, 0, (size_t)m * (size_t)n * (out_dtype == FP4Q_OUT_F32 ? 4u : 2u), s) == cudaSuccess
                   ? FP4Q_OK
                   : FP4Q_ERR_CUDA;
    if (!codes_a || !codes_b || !scales_a || !scales_b) return FP4Q_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(codes_a) & 15u) || (reinterpret_cast<uintptr_t>(codes_b) & 15u) ||
        (reinterpret_cast<uintptr_t>(scales_a) & 3u) || (reinterpret_cast<uintptr_t>(scales_b) & 3u))
        return FP4Q_ERR_ALIGN;
    f8gemm::Params p;
    memset(&p, 0, sizeof(p));
    if (!make_byte_map(&p.ta, codes_a, m, k, f8gemm::BM)) return FP4Q_ERR_CUDA;
    p.sa = scales_a;
    p.sb = scales_b;
    p.y = y;
    p.m = m;
    p.n = n;
    p.kb = (k + 127) / 128;
    p.f32 = out_dtype == FP4Q_OUT_F32;
    p.fault = device_fault_word();
    if (!p.fault) return FP4Q_ERR_CUDA;
    // Which kernel, by the times measured on 12 shapes (n 3584 to 13824, k 5120 and 18944, m 100 to 1024): a tile of
    // 128 x 256 takes 0.59 us a block of k, one of 128 x 128 0.32, both after 3 us; a CTA of the few-token kernel 0.38
    // after 10.  Up to 64 rows B's bytes bound the product and the few-token kernel, with all SMs, always leads
    // (37 x 3584 x 18944: 18 against 67 us); at 256 x 5120 x 5120 it takes 24.8 us, tiles of 128 x 128 take 15.8.
    // That holds within 10 % where the rows begin on 128-byte lines and y takes whole stores (200 x 3584 x 18944: 50
    // by the rule, 46 measured; 777 x 1024 x 4096: 13.2 and 13.1); an odd n adds 2 us there, k = 4112 another 3, so
    // that 777 x 1001 x 4112 takes 18.5 us where the rule says 13.6 and the few-token kernel would take 17.1.
    const int64_t tiles_m = (m + 127) / 128;
    const int64_t waves128 = (tiles_m * ((n + 127) / 128) + 147) / 148, waves256 = (tiles_m * ((n + 255) / 256) + 147) / 148;
    const int64_t ns128 = 3000 + 320 * p.kb * waves128, ns256 = 3000 + 590 * p.kb * waves256;
    const int ntok = m <= 16 ? 16 : m <= 32 ? 32 : 64;
    const int max_kb = ntok == 16 ? f8gemm::Small<16>::MAX_KB : ntok == 32 ? f8gemm::Small<32>::MAX_KB : f8gemm::Small<64>::MAX_KB;
    const int64_t tiles = ((m + ntok - 1) / ntok) * ((n + 127) / 128);
    const int split = f8gemm::split_of(tiles, p.kb, max_kb);
    if (split && (m <= 64 || (tiles * split <= 2 * 148 && 10000 + 380 * ((p.kb + split - 1) / split) < (ns128 < ns256 ? ns128 : ns256)))) {
        if (ntok == 16) return f8gemm::launch_small<16>(p, codes_a, codes_b, k, split, s);
        if (ntok == 32) return f8gemm::launch_small<32>(p, codes_a, codes_b, k, split, s);
        return f8gemm::launch_small<64>(p, codes_a, codes_b, k, split, s);
    }
    if (ns256 <= ns128) return f8gemm::launch<256>(p, codes_b, k, s);
    return f8gemm::launch<128>(p, codes_b, k, s);
}

// fp4q_f8.cu -- E4M3 quantizer with one fp32 scale per 128 values.
//
//   s = fp32(amax / 448) (1 when amax = 0),   code = e4m3(fp32(x / s)), RNE,
// amax over 1 x 128 elements of a row (activations) or a 128 x 128 tile
// (weights).  amax is taken on the integer patterns of |x|, so an infinity or
// NaN in a group reaches its scale and from there every value, as in the
// formula.  The quotient is the correctly rounded one without a division per
// element (div2_cr); scales outside its range divide.
//
// One pass: 2 bytes read and 1 written per value, the values stay in registers
// between the maximum and the codes, so memory bounds both kernels.  Measured
// (graph replays): 8192 x 5120 by rows 23.0 us, 5.5 TB/s (one load in flight per
// lane 23.7, two 23.0, four 26.8: fewer warps fit); 13824 x 5120 by tiles 35.5 us,
// 6.0 TB/s.
#include <cuda_runtime.h>

#include "fp4q_device.cuh"
#include "fp4q_launch.h"
#include "../../include/fp4q.h"

namespace fp4q {
namespace f8 {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int VEC = 16;                       // values per lane and load: 32 bytes in, 16 bytes out
constexpr int LANES = 128 / VEC;              // lanes of one group of 128

struct Params {
    const uint16_t* x;
    uint8_t* codes;
    float* scales;
    int64_t rows, cols, groups;               // groups: of 128 columns, all rows
    int64_t kb;                               // groups per row
};

// Pattern of the largest |x| among 16 bf16 values (NaN above infinity above the rest).
__device__ __forceinline__ uint32_t amax16(const U32x8& w)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w.v[i] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
}

// fp32(amax / 448) from the bf16 pattern of amax.
__device__ __forceinline__ float scale_of(uint32_t amax_bits)
{
    return amax_bits == 0u ? 1.0f : __fdiv_rn(as_f32(amax_bits << 16), 448.0f);
}

__device__ __forceinline__ uint32_t e4m3_pack4(f32x2 a, f32x2 b)
{
    float a0, a1, b0, b1;
    upk(a, a0, a1);
    upk(b, b0, b1);
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
    return r;
}

// Codes of 16 values under scale s (the quotients are at most 448 (1 + 2^-8),
// which rounds to 448: nothing saturates).
__device__ __forceinline__ void encode16(const U32x8& w, float s, uint32_t (&out)[4])
{
    if (s >= kDivLo && s <= kDivHi) {
        const float r = __frcp_rn(s);
        const f32x2 R = pk(r, r), nS = pk(-s, -s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = w.v[2 * i], b = w.v[2 * i + 1];
            out[i] = e4m3_pack4(div2_cr(pk(bf16_lo(a), bf16_hi(a)), R, nS), div2_cr(pk(bf16_lo(b), bf16_hi(b)), R, nS));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = w.v[2 * i], b = w.v[2 * i + 1];
            out[i] = e4m3_pack4(pk(__fdiv_rn(bf16_lo(a), s), __fdiv_rn(bf16_hi(a), s)),
                                pk(__fdiv_rn(bf16_lo(b), s), __fdiv_rn(bf16_hi(b), s)));
        }
    }
}

// 1 x 128 groups: 8 lanes per group, 4 groups per warp and load, U loads in
// flight per lane (one for small tensors, so that more SMs take part).
template <int U>
__global__ void __launch_bounds__(THREADS) f8_rows_kernel(const Params p)
{
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    const int sub = lane / LANES, at = (lane % LANES) * VEC;
    const int64_t g0 = warp * (4 * U) + sub;
    U32x8 w[U];
    int64_t off[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t g = g0 + 4 * u;
        off[u] = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[u].v[i] = 0u;
        if (g < p.groups) {
            int64_t row;
            if ((uint64_t)p.groups < (1ull << 32))
                row = (uint32_t)g / (uint32_t)p.kb;
            else
                row = g / p.kb;
            const int64_t col = (g - row * p.kb) * 128 + at;
            if (col < p.cols) {                              // the last group of a row may be short
                off[u] = row * p.cols + col;
                w[u] = ldg256_stream(p.x + off[u]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t m = amax16(w[u]);
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float s = scale_of(m);
        if (off[u] >= 0) {
            uint32_t c[4];
            encode16(w[u], s, c);
            stg128(p.codes + off[u], c[0], c[1], c[2], c[3]);
            if (at == 0) p.scales[g0 + 4 * u] = s;
        }
    }
}

// 128 x 128 tiles: one CTA per tile, 16 rows per warp, 4 rows per load.
__global__ void __launch_bounds__(THREADS) f8_tiles_kernel(const Params p)
{
    pdl_wait();
    pdl_release();
    __shared__ uint32_t part[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tr = blockIdx.x / p.kb, tc = blockIdx.x - tr * p.kb;
    const int64_t col = tc * 128 + (lane % LANES) * VEC;
    const int64_t row0 = tr * 128 + warp * 16 + lane / LANES;
    U32x8 w[4];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[u].v[i] = 0u;
        if (col < p.cols && row0 + 4 * u < p.rows) w[u] = ldg256_stream(p.x + (row0 + 4 * u) * p.cols + col);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) m = max(m, amax16(w[u]));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) part[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WARPS; ++i) m = max(m, part[i]);
    const float s = scale_of(m);
    if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (col < p.cols && row0 + 4 * u < p.rows) {
            uint32_t c[4];
            encode16(w[u], s, c);
            stg128(p.codes + (row0 + 4 * u) * p.cols + col, c[0], c[1], c[2], c[3]);
        }
}

}  // namespace f8
}  // namespace fp4q

extern "C" int fp4q_f8_quantize(const void* x, int64_t rows, int64_t cols, int grain, uint8_t* codes, float* scales,
                                void* stream)
{
    using namespace fp4q;
    if (rows < 0 || cols < 0 || cols % 16 != 0) return FP4Q_ERR_SHAPE;
    if (grain != FP4Q_F8_ROW && grain != FP4Q_F8_TILE) return FP4Q_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return FP4Q_OK;
    if (rows > INT64_MAX / 4 / cols) return FP4Q_ERR_SHAPE;
    const int64_t kb = (cols + 127) / 128;
    const int64_t tiles = ((rows + 127) / 128) * kb;
    // one CTA per tile, or per 32 groups at least: the grid's x extent is 2^31 - 1
    if (tiles > INT32_MAX || rows > (int64_t)INT32_MAX * 32 / kb) return FP4Q_ERR_SHAPE;
    if (!x || !codes || !scales) return FP4Q_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(x) & 31u) || (reinterpret_cast<uintptr_t>(codes) & 15u) ||
        (reinterpret_cast<uintptr_t>(scales) & 3u))
        return FP4Q_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    f8::Params p{static_cast<const uint16_t*>(x), codes, scales, rows, cols, rows * kb, kb};
    cudaError_t e;
    if (grain == FP4Q_F8_TILE)
        e = launch_pdl(f8::f8_tiles_kernel, (int)tiles, f8::THREADS, 0, s, p);
    else if (p.groups <= 148 * 64)
        e = launch_pdl(f8::f8_rows_kernel<1>, (int)((p.groups + 31) / 32), f8::THREADS, 0, s, p);
    else
        e = launch_pdl(f8::f8_rows_kernel<2>, (int)((p.groups + 63) / 64), f8::THREADS, 0, s, p);
    return e == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

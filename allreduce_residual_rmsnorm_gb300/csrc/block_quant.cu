// Block quantisation to FP8 E4M3 with an fp32 scale per 128 elements, after an
// optional gated activation, written to one or several rows.
//
// A thread holds 16 elements of a row, 8 threads a block: the block's amax is
// three shuffles, the codes leave as one 128-bit store.  Each input element is
// read once, quantised once, and written `copies` times.  Without the activation
// memory bounds it (4096 x 7168 bf16 into 8 copies 46.8 us, 6.4 TB/s; 8192 x 7168
// fp32 44.8, 6.6; 16384 x 7168 bf16 59.5, 6.0); with it its instructions and the latency of the loads do
// (16384 x 2048: 29.9 us, 5.65 TB/s; with log2 e in one part 29.0, then 29.8
// without the bound on registers and 30.9 in blocks of 256).  Blocks that stay and load their next item ahead gained 3%
// there and lost 13% at 128 rows in 8 copies, and were not kept.
#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kThreads = 128;
constexpr int kElems = 16;      // per thread
constexpr float kFp8Max = 448.0f;

// the largest magnitude of three; NaN is passed over, or wins with `_nan`
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_abs3_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two of g / (1 + e^-g) * u for |g| < kPlainGate, where everything stays finite.
// e^-g = 2^t, t = -g log2 e: log2 e in two parts (Cody and Waite, Software Manual
// for the Elementary Functions, 1980), the rounding error of the product with
// the high part recovered by a fused multiply-add, so that t = -(minus_t - err)
// with err below 2^-17.  e^-g is then p + p err ln 2 with p = 2^-minus_t.  One
// part alone is off by 1.9e-8 |g| in t, 22 u at g = -87 (u = 2^-24).
// The quotient is G / d with G = g / 4 and d = (1 + e^-g) / 4 (a quarter, so that
// the reciprocal is not below the normal range), by the approximate reciprocal (1
// ulp) and one correction.  d is added up from its smaller parts, without
// rounding e^-g by itself.
// Off by at most: ex2 2.45 u (measured over every argument), the sum d, the
// quotient and the product with u one u each: 5.5 u.  In packed pairs: with expf
// and the divide instructions 32 a element, which bound the kernel (38.5 us at
// 16384 x 2048).
constexpr float kPlainGate = 88.0f;

__device__ __forceinline__ uint64_t silu_mul_pair(uint64_t g, uint64_t u)
{
    const float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const uint64_t quarter = pair_of(0.25f, 0.25f), minus_quarter = pair_of(-0.25f, -0.25f);
    const uint64_t minus_t = mul_pair(g, pair_of(kLog2e, kLog2e));
    // minus_t - g log2 e, exact but for the low part's own rounding
    const uint64_t err = fma3_pair(g, pair_of(-kLog2eLow, -kLog2eLow),
                                   fma3_pair(g, pair_of(-kLog2e, -kLog2e), minus_t));
    const float2 tf = unpack_pair(minus_t);
    float2 p, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(-tf.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(-tf.y));
    const uint64_t pp = pair_of(p.x, p.y);
    const uint64_t G = mul_pair(g, quarter);
    // -d = -p / 4 + (-1 / 4 - p err ln 2 / 4)
    const uint64_t low = fma3_pair(pp, mul_pair(err, pair_of(-0.25f * kLn2, -0.25f * kLn2)),
                                   minus_quarter);
    const uint64_t minus_d = fma3_pair(pp, minus_quarter, low);
    const float2 df = unpack_pair(minus_d);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-df.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-df.y));
    const uint64_t rr = pair_of(r.x, r.y);
    const uint64_t q = mul_pair(G, rr);
    const uint64_t rem = fma3_pair(q, minus_d, G);
    return mul_pair(fma3_pair(rem, rr, q), u);
}

// the same of one pair of numbers, for any gate
__device__ __noinline__ float silu_mul(float g, float u)
{
    return g / (1.0f + expf(-g)) * u;
}

template <class D, bool ACT>
__global__ void __launch_bounds__(kThreads, D::bytes == 4 ? 10 : 12)
    block_quant_kernel(BlockQuantArgs a, int chunks)
{
    // one item = 8 threads = one block of 128 of one row; `chunks` blocks per row
    // (32 bits: 2^31 items would be 275 GB of codes)
    const uint32_t item = blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3);
    const int sub = threadIdx.x & 7;
    const uint64_t row = item / (unsigned)chunks;
    const int blk = (int)(item - (uint32_t)row * (unsigned)chunks);
    const int at = blk * AR_QUANT_BLOCK + sub * kElems;
    pdl_trigger();
    pdl_wait();
    uint64_t rows = (uint64_t)a.rows;
    if (a.row_count)
        rows = (uint64_t)min(max(*a.row_count, 0), a.rows);
    const bool live = row < rows;
    const bool have = live && at < a.hidden;    // hidden % 16 == 0: all 16 or none
    float y[kElems];
#pragma unroll
    for (int i = 0; i < kElems; ++i)
        y[i] = 0.0f;
    if (have) {
        const uint64_t pitch = (uint64_t)a.hidden * (ACT ? 2 : 1) * D::bytes;
        const uint8_t* p = a.in + row * pitch + (uint64_t)at * D::bytes;
        typename D::Vec v[2], u[2];
        v[0] = load8_raw<D>(p);
        v[1] = load8_raw<D>(p + 8 * D::bytes);
        if constexpr (ACT) {
            const uint8_t* q = p + (uint64_t)a.hidden * D::bytes;
            u[0] = load8_raw<D>(q);
            u[1] = load8_raw<D>(q + 8 * D::bytes);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
            unpack8<D>(v[h], f);
            if constexpr (ACT) {
                float g[8];
                unpack8<D>(u[h], g);
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    top = max_abs3_nan(top, f[i], f[i + 1]);
                if (top < kPlainGate) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 o = unpack_pair(silu_mul_pair(pair_of(f[i], f[i + 1]),
                                                                   pair_of(g[i], g[i + 1])));
                        f[i] = o.x;
                        f[i + 1] = o.y;
                    }
                } else {
                    // a gate that is no number or far out
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = silu_mul(f[i], g[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[8 * h + i] = f[i];
        }
    }
    float amax = 0x1p-100f;     // NaN is passed over
#pragma unroll
    for (int i = 0; i < kElems; i += 2)
        amax = max_abs3(amax, y[i], y[i + 1]);
#pragma unroll
    for (int m = 4; m >= 1; m >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const float inv = __fdiv_rn(kFp8Max, amax);
    const float scale = __fdiv_rn(amax, kFp8Max);
    if (!have)
        return;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = y[i] * inv;
        hi[i] = y[8 + i] * inv;
    }
    const uint2 c0 = e4m3x8(lo), c1 = e4m3x8(hi);
    const uint4 codes = make_uint4(c0.x, c0.y, c1.x, c1.y);
    for (int j = 0; j < a.copies; ++j) {
        int64_t to = (int64_t)row;
        if (a.position)
            to = a.position[row * a.copies + j];
        if (to < 0 || to >= a.out_rows)
            continue;
        st_vec(a.q + (uint64_t)to * a.hidden + at, codes);
        if (sub == 0)
            a.scale[(uint64_t)to * chunks + blk] = scale;
    }
}

template <class D>
cudaError_t launch_t(const BlockQuantArgs& a, cudaStream_t s)
{
    const int chunks = quant_blocks(a.hidden);
    const uint64_t items = (uint64_t)a.rows * chunks;
    if (items > 0x7fffff00ull)
        return cudaErrorInvalidValue;
    const uint64_t blocks = (items * 8 + kThreads - 1) / kThreads;
    if (a.act == AR_ACT_SILU_MUL)
        return launch_after(block_quant_kernel<D, true>, (unsigned)blocks, kThreads, 0, s, a, chunks);
    return launch_after(block_quant_kernel<D, false>, (unsigned)blocks, kThreads, 0, s, a, chunks);
}

}  // namespace

cudaError_t launch_block_quant(int dtype, const BlockQuantArgs& a, cudaStream_t s)
{
    switch (dtype) {
    case AR_DT_BF16: return launch_t<Bf16>(a, s);
    case AR_DT_FP16: return launch_t<Fp16>(a, s);
    default: return launch_t<F32>(a, s);
    }
}

}  // namespace arf

// Block quantisation to FP8 E4M3 with an fp32 scale per 128 elements, after an
// optional gated activation, written to one or several rows.
//
// A thread holds 16 elements of a row, 8 threads a block: the block's amax is
// three shuffles, the codes leave as one 128-bit store.  Bounded by memory:
// each input element is read once, quantised once, and written `copies` times.
#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kThreads = 256;
constexpr int kElems = 16;      // per thread
constexpr float kFp8Max = 448.0f;

template <class D, bool ACT>
__global__ void __launch_bounds__(kThreads) block_quant_kernel(BlockQuantArgs a, int chunks)
{
    // one item = 8 threads = one block of 128 of one row; `chunks` blocks per row
    const uint64_t item = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) >> 3;
    const int sub = threadIdx.x & 7;
    const uint64_t row = item / (unsigned)chunks;
    const int blk = (int)(item - row * (unsigned)chunks);
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
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = f[i] / (1.0f + expf(-f[i])) * g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[8 * h + i] = f[i];
        }
    }
    float amax = 0x1p-100f;     // fmaxf passes over NaN
#pragma unroll
    for (int i = 0; i < kElems; ++i)
        amax = fmaxf(amax, fabsf(y[i]));
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
    const uint64_t threads = (uint64_t)a.rows * chunks * 8;
    const uint64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffull)
        return cudaErrorInvalidValue;
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

// Product of FP8 E4M3 matrices with an fp32 scale per block of 128, dense or
// by experts: out = sum over blocks of sa * sb * (a . b), in fp32.
//
// A 64 x 64 tile per thread block, 4 x 4 outputs per thread, 32 of the depth
// at a time through shared memory as fp32.
#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kTile = 64, kStep = 32;

template <class D>
__device__ __forceinline__ void store1(void* out, uint64_t i, float v)
{
    if constexpr (D::bytes == 4)
        static_cast<float*>(out)[i] = v;
    else if constexpr (D::id == AR_DT_BF16)
        static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(out)[i] = __float2half_rn(v);
}

template <class D>
__global__ void __launch_bounds__(256) matmul_kernel(MatmulArgs a)
{
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    const int e = blockIdx.z;
    int row0 = 0, row1 = a.rows;
    if (a.offsets) {
        row0 = min(max(a.offsets[e], 0), a.rows);
        row1 = min(max(a.offsets[e + 1], row0), a.rows);
    }
    const int nb = (a.depth + AR_QUANT_BLOCK - 1) / AR_QUANT_BLOCK;
    const int ncb = (a.cols + AR_QUANT_BLOCK - 1) / AR_QUANT_BLOCK;
    const int n0 = blockIdx.x * kTile;
    const uint8_t* b = a.b + (uint64_t)e * a.cols * a.depth;
    const float* sb = a.sb + ((uint64_t)e * ncb + n0 / AR_QUANT_BLOCK) * nb;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t m0 = row0 + (int64_t)blockIdx.y * kTile; m0 < row1;
         m0 += (int64_t)gridDim.y * kTile) {
        float acc[4][4] = {};
        for (int kb = 0; kb < nb; ++kb) {
            float part[4][4] = {};
            const int kend = min(a.depth, (kb + 1) * AR_QUANT_BLOCK);
            for (int k0 = kb * AR_QUANT_BLOCK; k0 < kend; k0 += kStep) {
                __syncthreads();
                for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
                    const int r = i / kStep, k = i % kStep;
                    const bool in = k0 + k < kend;
                    as[k][r] = in && m0 + r < row1
                                   ? e4m3_to_f32(a.a[(uint64_t)(m0 + r) * a.depth + k0 + k])
                                   : 0.0f;
                    bs[k][r] = in && n0 + r < a.cols
                                   ? e4m3_to_f32(b[(uint64_t)(n0 + r) * a.depth + k0 + k])
                                   : 0.0f;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kStep; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part[i][j] = fmaf(as[k][ty + 16 * i], bs[k][tx + 16 * j], part[i][j]);
            }
            const float sbk = sb[kb];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + ty + 16 * i;
                const float s = m < row1 ? a.sa[(uint64_t)m * nb + kb] * sbk : 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i;
                const int n = n0 + tx + 16 * j;
                if (m < row1 && n < a.cols)
                    store1<D>(a.out, (uint64_t)m * a.cols + n, acc[i][j]);
            }
    }
}

}  // namespace

cudaError_t launch_matmul(int dtype, const MatmulArgs& a, cudaStream_t s)
{
    const int per = (a.rows + a.experts - 1) / a.experts;
    const int my = (per + kTile - 1) / kTile;
    const dim3 grid((a.cols + kTile - 1) / kTile, my > 1024 ? 1024 : my, a.experts);
    switch (dtype) {
    case AR_DT_BF16: matmul_kernel<Bf16><<<grid, 256, 0, s>>>(a); break;
    case AR_DT_FP16: matmul_kernel<Fp16><<<grid, 256, 0, s>>>(a); break;
    default: matmul_kernel<F32><<<grid, 256, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace arf

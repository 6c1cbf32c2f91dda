// Weighted combination of expert rows back to token rows: 8 elements of one
// token per thread, the rows of up to 8 experts loaded before the first is
// used.  Bounded by memory: every expert row is read once, fp32 sums in slot
// order, one rounding.
#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;       // rows in flight per thread

template <class D>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a, int vecs)
{
    const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const uint64_t t = i / (unsigned)vecs;
    pdl_trigger();
    pdl_wait();
    if (t >= (uint64_t)a.T)
        return;
    const uint64_t at = (i - t * (unsigned)vecs) * 8 * D::bytes;
    const uint64_t pitch = (uint64_t)a.H * D::bytes;
    float s[8];
    if (a.add) {
        unpack8<D>(load8_raw<D>(a.add + t * pitch + at), s);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[e] = 0.0f;
    }
    const int32_t* pos = a.position + t * a.k;
    const float* wt = a.weights + t * a.k;
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
        typename D::Vec v[kAhead];
        float w[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            on[j] = false;
            if (j0 + j < a.k) {
                const int32_t p = pos[j0 + j];
                on[j] = p >= 0 && p < a.in_rows;
                if (on[j]) {
                    w[j] = wt[j0 + j];
                    v[j] = load8_raw<D>(a.rows + (uint64_t)p * pitch + at);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (on[j]) {
                float f[8];
                unpack8<D>(v[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] = fmaf(w[j], f[e], s[e]);
            }
        }
    }
    store8<D>(a.out + t * pitch + at, s);
}

template <class D>
cudaError_t launch_t(const CombineArgs& a, cudaStream_t s)
{
    const int vecs = a.H / 8;
    const uint64_t blocks = ((uint64_t)a.T * vecs + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffull)
        return cudaErrorInvalidValue;
    return launch_after(combine_kernel<D>, (unsigned)blocks, kThreads, 0, s, a, vecs);
}

}  // namespace

cudaError_t launch_combine(int dtype, const CombineArgs& a, cudaStream_t s)
{
    switch (dtype) {
    case AR_DT_BF16: return launch_t<Bf16>(a, s);
    case AR_DT_FP16: return launch_t<Fp16>(a, s);
    default: return launch_t<F32>(a, s);
    }
}

}  // namespace arf

// Attention of prompts (any number of new tokens per sequence) over the paged cache.
//
// A warp has one row and query head, a lane four elements of the head; keys one
// after the other with a running maximum and sum.  The simplest form that is right.
#include "ar_internal.h"
#include "attention_internal.h"
#include "expert_vec.cuh"
#include "matmul_internal.h"

namespace arf {
namespace {

constexpr int kThreads = 256;

template <class D>
__global__ void __launch_bounds__(kThreads) prompt_attention_kernel(AttentionArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    const int row = (int)(item / a.Hq), h = (int)(item - (int64_t)row * a.Hq);
    if (row >= a.T)
        return;
    int seq = -1;
    for (int s0 = 0; s0 <= a.c.S; s0 += 32)
        seq += __reduce_add_sync(0xffffffffu, s0 + lane <= a.c.S && a.starts[s0 + lane] <= row);
    if (seq < 0 || seq >= a.c.S || a.starts[seq] < 0 || a.starts[seq + 1] <= row || a.starts[seq + 1] > a.T)
        return;
    const int i = clamp_length(a.c, a.c.lengths[seq]) - (a.starts[seq + 1] - row);
    const int low = a.window ? i - a.window + 1 : 0, hk = h / a.G;
    float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    for (int e = 0; e < 4; ++e)
        q[e] = 4 * lane + e < a.c.D
                   ? load1<D>(a.q.p + row * a.q.row + h * a.q.head, 4 * lane + e) * a.scale_log2
                   : 0.0f;
    for (int j = 0; j <= i; ++j) {
        if (j < low && j >= a.sinks) {
            j = low - 1;
            continue;
        }
        const int page = a.c.table[(int64_t)seq * a.c.max_pages + (j >> a.c.page_shift)];
        const int in = j & ((1 << a.c.page_shift) - 1);
        const bool there = page >= 0 && page < a.c.pages;
        float s = 0.0f;
        for (int e = 0; e < 4; ++e)
            if (there && 4 * lane + e < a.c.D)
                s = fmaf(q[e], load1<D>(a.c.k + page * a.c.k_page + in * a.c.k_row + hk * a.c.k_head,
                                        4 * lane + e), s);
        for (int k = 1; k < 32; k <<= 1)
            s += __shfl_xor_sync(0xffffffffu, s, k);
        const float top = fmaxf(m, s), base = top == -INFINITY ? 0.0f : top;
        const float f = exp2f(m - base), p = exp2f(s - base);
        l = fmaf(l, f, p);
        for (int e = 0; e < 4; ++e) {
            o[e] *= f;
            if (there && 4 * lane + e < a.c.D)
                o[e] = fmaf(p, load1<D>(a.c.v + page * a.c.v_page + in * a.c.v_row + hk * a.c.v_head,
                                        4 * lane + e), o[e]);
        }
        m = top;
    }
    for (int e = 0; e < 4; ++e)
        if (4 * lane + e < a.c.D)
            reinterpret_cast<uint16_t*>(a.out.p + row * a.out.row + h * a.out.head)[4 * lane + e] =
                (uint16_t)pack2<D>(l == 0.0f ? 0.0f : o[e] / l, 0.0f);
    if (a.lse && lane == 0)
        a.lse[(int64_t)row * a.Hq + h] = (m + log2f(l)) * 0.693147181f;
}

}  // namespace

cudaError_t launch_prompt_attention(int dtype, const AttentionArgs& a, cudaStream_t s)
{
    const int64_t blocks = ((int64_t)a.T * a.Hq + kThreads / 32 - 1) / (kThreads / 32);
    return dtype == AR_DT_BF16
               ? launch_after(prompt_attention_kernel<Bf16>, (unsigned)blocks, kThreads, 0, s, a)
               : launch_after(prompt_attention_kernel<Fp16>, (unsigned)blocks, kThreads, 0, s, a);
}

}  // namespace arf

extern "C" int ar_fusion_attention_status(void* stream, int* detail)
{
    (void)stream;
    if (detail)
        *detail = -1;
    return AR_OK;
}

// Launchers behind the attention-layer entry points (not part of the C ABI).
// Each returns the cudaError_t of its launch; arguments are already checked.
#pragma once

#include <mutex>

#include "expert_internal.h"

namespace arf {

// ar_kv_cache with strides in bytes; that of an extent of one is 0
struct CacheArgs {
    uint8_t *k, *v;
    int64_t k_page, k_row, k_head, v_page, v_row, v_head;
    int pages, page_shift, heads, D, S, max_pages;
    const float* scale;             // [2] or NULL
    const int32_t* table;
    const int32_t* lengths;
};
// ar_head_rows with strides in bytes
struct Rows {
    uint8_t* p;
    int64_t row, head;
};

struct RopeArgs {
    CacheArgs c;
    Rows q, q_out, k, v;            // q.p NULL: keys and values alone
    int T, Hq, rot, interleaved, axes;
    const int32_t* starts;
    const int32_t* positions;
    const float* inv_freq;
    int ends[AR_MAX_AXES];          // pairs before the end of each axis
};
cudaError_t launch_rope_append(int dtype, bool e4m3, const RopeArgs& a, cudaStream_t s);

struct AttentionArgs {
    CacheArgs c;
    Rows q, out;
    float* lse;                     // [rows][Hq] or NULL
    const int32_t* starts;          // prompts only
    int T, Hq, G;                   // G query heads share a head of the cache
    float scale_log2;               // scale * log2 e
    int window, sinks;              // window 0: every key
    uint8_t* work;
    uint64_t work_bytes;
};
cudaError_t launch_decode_attention(int dtype, bool e4m3, const AttentionArgs& a, cudaStream_t s);
cudaError_t launch_prompt_attention(int dtype, bool e4m3, const AttentionArgs& a, cudaStream_t s);
// Held over the two launches of a call that is split.  Threads that call on one stream may share a
// workspace; another's kernel between this one's and its join would overwrite the pieces, and each
// join would add up what it finds, with the sizes of its own call.  A lock for the workspace's
// address: calls with workspaces of their own seldom meet.
std::mutex& launches_with(const void* workspace);

// Unit `in` of a list of items of n units each.  The units of one sequence's items pass 2^31 (at
// 2^30 tokens and 128 heads), its items and the units of one do not.
struct UnitPlace {
    int item, unit;
};
__host__ __device__ inline UnitPlace unit_place(long long in, int n)
{
    if (in >> 31 == 0)
        return UnitPlace{(int)((unsigned)in / (unsigned)n), (int)((unsigned)in % (unsigned)n)};
    return UnitPlace{(int)(in / n), (int)(in % n)};
}

// tokens of a sequence that the table can hold
__device__ __forceinline__ int clamp_length(const CacheArgs& c, int length)
{
    return min(max(length, 0), c.max_pages << c.page_shift);
}

}  // namespace arf

// Launchers behind the attention-layer entry points (not part of the C ABI).
// Each returns the cudaError_t of its launch; arguments are already checked.
#pragma once

#include <string.h>

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

// Units of a prompt's item of so many steps in the list that the blocks share equally.  Its end, the
// output and masks, takes as long as two steps: with the steps alone the block that had the list's
// last items, of one or two steps each, was the last by far (a prompt of 3000 tokens, 32 / 8 heads,
// 121 us instead of 78, 60 x 4 new tokens on 500-32000, 64 / 8 heads, 376 instead of 306; one
// unit 84 and 322, three 79 and 303).
constexpr int kItemEnd = 2;
__host__ __device__ inline int share_of(int steps) { return steps ? steps + kItemEnd : 0; }

// The angle position * f as a fixed-point part of a turn: f / (2 pi), less its whole turns, times
// 2^64.  A position times that, in 64 bits that wrap, loses whole turns exactly, and what the last
// bits lack is position * 2^-62 of a turn at most (times f, where that is above 1): as exact at any
// position as at 1.  (With f / pi in two floats, reduced in two parts, 2^-18 of half a turn were
// lost at positions near 2^31; 8192 rows took 35.8 us and take 36.3.)
__host__ __device__ inline uint64_t turns_of(float f)
{
    constexpr uint64_t kInverse = 0x28be60db9391054aull;        // 2^64 / (2 pi)
    uint32_t bits;
    memcpy(&bits, &f, 4);
    // |f| = m 2^(e - 23) for e <= 0, and what is below the normal range is no turn
    const int e = (int)(bits >> 23 & 0xff) - 127;
    const uint64_t m = (bits & 0x7fffff) | 0x800000;
    // m * kInverse / 2^23
    const uint64_t x = (m * (kInverse >> 32) << 9) + (m * (kInverse & 0xffffffffu) >> 23);
    const uint64_t t = e <= 0 ? x >> (-e < 63 ? -e : 63) : x << (e < 63 ? e : 63);
    return bits >> 31 ? 0 - t : t;
}
// position * f / pi in [-1, 1], rounded to a float once
__host__ __device__ inline float half_turns(int position, uint64_t turns)
{
    return (float)(int64_t)((uint64_t)(int64_t)position * turns) * 0x1p-63f;
}

// tokens of a sequence that the table can hold
__device__ __forceinline__ int clamp_length(const CacheArgs& c, int length)
{
    return min(max(length, 0), c.max_pages << c.page_shift);
}

}  // namespace arf

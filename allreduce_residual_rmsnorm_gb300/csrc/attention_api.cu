// C ABI of the attention-layer calls: argument checks and dispatch.  The contract
// of every entry point is in include/ar_fusion.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "ar_internal.h"
#include "attention_internal.h"

using namespace arf;

namespace {

int afail(int code, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_last_error(code, buf);
}

int launched(cudaError_t e, const char* what)
{
    if (e != cudaSuccess)
        return afail(AR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return AR_OK;
}

bool aligned(const void* p, unsigned to) { return p && ((uintptr_t)p & (to - 1)) == 0; }
bool aligned_or_null(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) == 0; }

// strides of pages, rows and heads in bytes
int cache_strides(const char* name, const ar_kv_cache& c, int64_t page, int64_t row, int64_t head,
                  int bytes, int64_t* out)
{
    const int64_t in[3] = {page, row, head};
    const int extent[3] = {c.pages, c.page_size, c.heads};
    for (int i = 0; i < 3; ++i) {
        out[i] = 0;
        if (extent[i] == 1)
            continue;
        if (in[i] < 1 || in[i] >= (int64_t)1 << 40 || in[i] * bytes % 16 != 0 ||
            in[i] * bytes >= (int64_t)1 << 40)
            return afail(AR_ERR_INVALID, "%s: stride %lld is not a positive multiple of 16 bytes below 2^40",
                         name, (long long)in[i]);
    }
    for (int i = 0; i < 3; ++i)
        out[i] = extent[i] == 1 ? 0 : in[i] * bytes;
    return AR_OK;
}

// dtype: that of the call's rows.  Pointers are looked at only where something runs.
int take_cache(const ar_kv_cache* cache, int dtype, bool runs, CacheArgs* a, bool* e4m3)
{
    if (!cache)
        return afail(AR_ERR_INVALID, "cache NULL");
    const ar_kv_cache& c = *cache;
    if (dtype != AR_DT_BF16 && dtype != AR_DT_FP16)
        return afail(AR_ERR_UNSUPPORTED, "dtype %d is not bf16 (0) or fp16 (1)", dtype);
    *e4m3 = c.dtype == AR_DT_E4M3;
    if (c.dtype != AR_DT_BF16 && c.dtype != AR_DT_FP16 && !*e4m3)
        return afail(AR_ERR_UNSUPPORTED, "cache dtype %d is not bf16 (0), fp16 (1) or E4M3 (3)",
                     c.dtype);
    if (!*e4m3 && c.dtype != dtype)
        return afail(AR_ERR_INVALID, "cache dtype %d is not that of the rows, %d", c.dtype, dtype);
    if (c.pages < 1 || c.heads < 1 || c.max_pages < 1 || c.sequences < 0)
        return afail(AR_ERR_INVALID, "pages %d, heads %d or max_pages %d < 1, or sequences %d < 0",
                     c.pages, c.heads, c.max_pages, c.sequences);
    if (c.page_size < 1 || (c.page_size & (c.page_size - 1)))
        return afail(AR_ERR_INVALID, "page_size %d is not a power of two", c.page_size);
    if (c.page_size < 8 || c.page_size > 65536)
        return afail(AR_ERR_UNSUPPORTED, "page_size %d outside 8..65536", c.page_size);
    if (c.sequences > AR_MAX_SEQUENCES)
        return afail(AR_ERR_UNSUPPORTED, "sequences %d > %d", c.sequences, AR_MAX_SEQUENCES);
    // ends of tiles of keys stay within 32 bits
    if ((int64_t)c.max_pages * c.page_size > INT_MAX - 1023)
        return afail(AR_ERR_UNSUPPORTED, "max_pages %d x page_size %d beyond 2^31 - 1024", c.max_pages,
                     c.page_size);
    const int unit = *e4m3 ? 16 : 8;
    if (c.head_dim < unit || c.head_dim % unit != 0)
        return afail(AR_ERR_INVALID, "head_dim %d is not a positive multiple of %d", c.head_dim, unit);
    if (c.head_dim > AR_MAX_HEAD_DIM)
        return afail(AR_ERR_UNSUPPORTED, "head_dim %d > %d", c.head_dim, AR_MAX_HEAD_DIM);
    if (c.scale && !*e4m3)
        return afail(AR_ERR_INVALID, "scale given with a cache of 16-bit elements");
    const int bytes = *e4m3 ? 1 : 2;
    int64_t k[3], v[3];
    int rc = cache_strides("k", c, c.k_page, c.k_row, c.k_head, bytes, k);
    if (rc == AR_OK)
        rc = cache_strides("v", c, c.v_page, c.v_row, c.v_head, bytes, v);
    if (rc != AR_OK)
        return rc;
    if (runs) {
        if (!aligned(c.k, 16) || !aligned(c.v, 16))
            return afail(AR_ERR_INVALID, "k or v of the cache NULL or not 16-byte aligned");
        if (!aligned(c.page_table, 4) || !aligned(c.lengths, 4) || !aligned_or_null(c.scale, 4))
            return afail(AR_ERR_INVALID, "page_table or lengths NULL, or one of them or scale misaligned");
    }
    int shift = 0;
    while (1 << shift < c.page_size)
        ++shift;
    *a = CacheArgs{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), k[0], k[1], k[2], v[0], v[1],
                   v[2], c.pages, shift, c.heads, c.head_dim, c.sequences, c.max_pages, c.scale,
                   c.page_table, c.lengths};
    return AR_OK;
}

// rows and heads: the extents
int take_rows(const char* name, const ar_head_rows* r, int rows, int heads, Rows* out)
{
    if (!r || !aligned(r->data, 16))
        return afail(AR_ERR_INVALID, "%s NULL or not 16-byte aligned", name);
    const auto bad = [](int64_t stride, int extent) {
        return extent > 1 && (stride < 1 || stride % 8 != 0 || stride >= (int64_t)1 << 39);
    };
    if (bad(r->row, rows) || bad(r->head, heads))
        return afail(AR_ERR_INVALID, "%s: strides %lld, %lld are not positive multiples of 16 bytes below 2^40",
                     name, (long long)r->row, (long long)r->head);
    *out = Rows{static_cast<uint8_t*>(r->data), rows > 1 ? 2 * r->row : 0, heads > 1 ? 2 * r->head : 0};
    return AR_OK;
}

int check_heads(int q_heads, int heads)
{
    if (q_heads < 1 || q_heads % heads != 0)
        return afail(AR_ERR_INVALID, "q_heads %d is not a positive multiple of the cache's heads %d",
                     q_heads, heads);
    return AR_OK;
}

int take_attention(const ar_kv_cache* cache, const ar_head_rows* q, const ar_head_rows* out,
                   float* lse, int tokens, int q_heads, int dtype, float scale, int window,
                   int sinks, void* workspace, size_t workspace_bytes, AttentionArgs* a, bool* e4m3)
{
    const bool runs = cache && cache->sequences > 0 && tokens > 0;
    int rc = take_cache(cache, dtype, runs, &a->c, e4m3);
    if (rc == AR_OK)
        rc = check_heads(q_heads, a->c.heads);
    if (rc != AR_OK)
        return rc;
    a->G = q_heads / a->c.heads;
    if (a->G > AR_MAX_HEAD_GROUP)
        return afail(AR_ERR_UNSUPPORTED, "%d query heads share a head: more than %d", a->G,
                     AR_MAX_HEAD_GROUP);
    if (!(scale > 0.0f) || !isfinite(scale) || !isfinite(scale * 1.44269504f))
        return afail(AR_ERR_INVALID, "scale %g is not positive and finite", scale);
    if (window < 0 || sinks < 0)
        return afail(AR_ERR_INVALID, "window %d or sinks %d < 0", window, sinks);
    if (sinks > 0 && window == 0)
        return afail(AR_ERR_INVALID, "sinks %d without a window", sinks);
    if (tokens > 0 && (int64_t)tokens * q_heads > INT_MAX)
        return afail(AR_ERR_UNSUPPORTED, "%d rows x %d heads beyond 2^31 - 1", tokens, q_heads);
    if (!aligned_or_null(workspace, 16) || (!workspace && workspace_bytes))
        return afail(AR_ERR_INVALID, "workspace NULL with %zu bytes, or not 16-byte aligned",
                     workspace_bytes);
    a->T = tokens;
    a->Hq = q_heads;
    a->lse = lse;
    a->starts = nullptr;
    a->scale_log2 = (float)((double)scale * 1.4426950408889634);
    // a window of all that the table holds is none
    const bool windowed = window > 0 && window < (int64_t)cache->max_pages * cache->page_size;
    a->window = windowed ? window : 0;
    a->sinks = windowed ? sinks : 0;
    a->work = static_cast<uint8_t*>(workspace);
    a->work_bytes = workspace_bytes;
    if (!runs)
        return AR_OK;
    if (!aligned_or_null(lse, 4))
        return afail(AR_ERR_INVALID, "lse misaligned");
    rc = take_rows("q", q, tokens, q_heads, &a->q);
    return rc == AR_OK ? take_rows("out", out, tokens, q_heads, &a->out) : rc;
}

}  // namespace

std::mutex& arf::launches_with(const void* workspace)
{
    static std::mutex locks[64];
    // the upper bits of a product with 2^64 over the golden ratio: neighbours far apart
    return locks[(uint64_t)(uintptr_t)workspace * 0x9e3779b97f4a7c15ull >> 58];
}

extern "C" {

int ar_fusion_rope_append(const ar_kv_cache* cache, const ar_head_rows* q,
                          const ar_head_rows* q_out, const ar_head_rows* k,
                          const ar_head_rows* v, int tokens, int q_heads, int dtype,
                          const int32_t* starts, const int32_t* positions,
                          const float* inv_freq, int rot, const int* sections, int axes,
                          int interleaved, void* stream)
{
    RopeArgs a = {};
    bool e4m3 = false;
    const bool runs = cache && cache->sequences > 0 && tokens > 0;
    int rc = take_cache(cache, dtype, runs, &a.c, &e4m3);
    if (rc != AR_OK)
        return rc;
    if (tokens < 0)
        return afail(AR_ERR_INVALID, "tokens %d < 0", tokens);
    if (!starts && tokens != cache->sequences)
        return afail(AR_ERR_INVALID, "tokens %d are not one for each of %d sequences, and starts is NULL",
                     tokens, cache->sequences);
    if (q && (rc = check_heads(q_heads, a.c.heads)) != AR_OK)
        return rc;
    // below 2^28 pieces of a row
    if ((q ? (int64_t)q_heads : 0) + 2 * (int64_t)a.c.heads >= 1 << 24)
        return afail(AR_ERR_UNSUPPORTED, "q_heads %d and twice heads %d beyond 2^24 - 1", q ? q_heads : 0,
                     a.c.heads);
    if (rot < 0 || rot % 16 != 0 || rot > a.c.D)
        return afail(AR_ERR_INVALID, "rot %d is not a multiple of 16 in 0..%d", rot, a.c.D);
    if (axes < 1 || axes > AR_MAX_AXES)
        return afail(AR_ERR_INVALID, "axes %d outside 1..%d", axes, AR_MAX_AXES);
    if (!sections && axes > 1)
        return afail(AR_ERR_INVALID, "sections NULL with %d axes", axes);
    int64_t sum = 0;
    for (int i = 0; i < axes; ++i) {
        const int n = sections ? sections[i] : rot / 2;
        if (n < 0)
            return afail(AR_ERR_INVALID, "sections[%d] %d < 0", i, n);
        sum += n;
        a.ends[i] = (int)(sum < rot / 2 ? sum : rot / 2);
    }
    if (sum != rot / 2)
        return afail(AR_ERR_INVALID, "sections add up to %lld, and rot / 2 is %d", (long long)sum,
                     rot / 2);
    if (interleaved != 0 && interleaved != 1)
        return afail(AR_ERR_INVALID, "interleaved %d is not 0 or 1", interleaved);
    if (!runs)
        return AR_OK;
    if (rot > 0 && !aligned(inv_freq, 4))
        return afail(AR_ERR_INVALID, "inv_freq NULL or misaligned");
    if (!aligned_or_null(starts, 4) || !aligned_or_null(positions, 4))
        return afail(AR_ERR_INVALID, "starts or positions misaligned");
    if (q && ((rc = take_rows("q", q, tokens, q_heads, &a.q)) != AR_OK ||
              (rc = take_rows("q_out", q_out, tokens, q_heads, &a.q_out)) != AR_OK))
        return rc;
    if ((rc = take_rows("k", k, tokens, a.c.heads, &a.k)) != AR_OK ||
        (rc = take_rows("v", v, tokens, a.c.heads, &a.v)) != AR_OK)
        return rc;
    a.T = tokens;
    a.Hq = q ? q_heads : 0;
    a.rot = rot;
    a.interleaved = interleaved;
    a.axes = axes;
    a.starts = starts;
    a.positions = positions;
    a.inv_freq = inv_freq;
    return launched(launch_rope_append(dtype, e4m3, a, static_cast<cudaStream_t>(stream)),
                    "rotation kernel launch");
}

int ar_fusion_decode_attention(const ar_kv_cache* cache, const ar_head_rows* q,
                               const ar_head_rows* out, float* lse, int q_heads, int dtype,
                               float scale, int window, int sinks, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    AttentionArgs a = {};
    bool e4m3 = false;
    const int rows = cache ? cache->sequences : 0;
    const int rc = take_attention(cache, q, out, lse, rows, q_heads, dtype, scale, window, sinks,
                                  workspace, workspace_bytes, &a, &e4m3);
    if (rc != AR_OK || rows == 0)
        return rc;
    return launched(launch_decode_attention(dtype, e4m3, a, static_cast<cudaStream_t>(stream)),
                    "decode attention launch");
}

int ar_fusion_prompt_attention(const ar_kv_cache* cache, const ar_head_rows* q,
                               const ar_head_rows* out, float* lse, const int32_t* starts,
                               int tokens, int q_heads, int dtype, float scale, int window,
                               int sinks, void* workspace, size_t workspace_bytes,
                               void* stream)
{
    AttentionArgs a = {};
    bool e4m3 = false;
    if (tokens < 0)
        return afail(AR_ERR_INVALID, "tokens %d < 0", tokens);
    const int rc = take_attention(cache, q, out, lse, tokens, q_heads, dtype, scale, window, sinks,
                                  workspace, workspace_bytes, &a, &e4m3);
    if (rc != AR_OK)
        return rc;
    if (cache->sequences == 0 || tokens == 0)
        return AR_OK;
    if (!aligned(starts, 4))
        return afail(AR_ERR_INVALID, "starts NULL or misaligned");
    a.starts = starts;
    return launched(launch_prompt_attention(dtype, e4m3, a, static_cast<cudaStream_t>(stream)),
                    "prompt attention launch");
}

}  // extern "C"

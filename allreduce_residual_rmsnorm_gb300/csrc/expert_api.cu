// C ABI of the expert-layer calls: argument checks and dispatch.  The contract
// of every entry point is in include/ar_fusion.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdarg.h>
#include <stdio.h>

#include "ar_internal.h"
#include "expert_internal.h"

using namespace arf;

namespace {

int efail(int code, const char* fmt, ...)
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
        return efail(AR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return AR_OK;
}

// longest row in blocks of AR_QUANT_BLOCK: the end of its last block fits 32 bits
constexpr int kMaxLength = INT_MAX - (AR_QUANT_BLOCK - 1);

bool aligned(const void* p, unsigned to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

int bad_dtype(int dtype)
{
    return efail(AR_ERR_UNSUPPORTED, "dtype %d is not bf16 (0), fp16 (1) or fp32 (2)", dtype);
}

int check_matmul(const MatmulArgs& m, int dtype)
{
    if (!dtype_supported(dtype))
        return bad_dtype(dtype);
    if (m.rows < 0 || m.cols < 1)
        return efail(AR_ERR_INVALID, "rows %d < 0 or cols %d < 1", m.rows, m.cols);
    if (m.depth < 16 || m.depth % 16 != 0)
        return efail(AR_ERR_INVALID, "depth %d is not a positive multiple of 16", m.depth);
    if (m.depth > kMaxLength)
        return efail(AR_ERR_UNSUPPORTED, "depth %d > %d", m.depth, kMaxLength);
    if (m.experts < 1)
        return efail(AR_ERR_INVALID, "experts %d < 1", m.experts);
    if (m.experts > AR_MAX_EXPERTS)
        return efail(AR_ERR_UNSUPPORTED, "experts %d > %d", m.experts, AR_MAX_EXPERTS);
    if ((long long)m.experts * m.cols > INT_MAX - 256 || m.rows > INT_MAX - 256)
        return efail(AR_ERR_UNSUPPORTED, "experts %d x cols %d or rows %d beyond 2^31 - 257",
                     m.experts, m.cols, m.rows);
    if (m.rows == 0)
        return AR_OK;
    if (!aligned(m.a, 16) || !aligned(m.b, 16) || !aligned(m.out, 16))
        return efail(AR_ERR_INVALID, "a, b or out NULL or not 16-byte aligned");
    if (!aligned(m.sa, 4) || !aligned(m.sb, 4))
        return efail(AR_ERR_INVALID, "a_scale or b_scale NULL or not 4-byte aligned");
    return AR_OK;
}

}  // namespace

extern "C" {

int ar_fusion_route(const void* logits, int tokens, int experts, int dtype, const float* bias,
                    int score, int groups, int groups_kept, int group_score, int topk,
                    int renormalize, float scale, int32_t* ids_out, float* weights_out,
                    void* stream)
{
    if (!dtype_supported(dtype))
        return bad_dtype(dtype);
    if (tokens < 0)
        return efail(AR_ERR_INVALID, "tokens %d < 0", tokens);
    if (experts < 1 || topk < 1 || groups < 1)
        return efail(AR_ERR_INVALID, "experts %d, topk %d or groups %d < 1", experts, topk, groups);
    if (experts > AR_MAX_EXPERTS || topk > AR_MAX_TOPK || groups > AR_MAX_GROUPS)
        return efail(AR_ERR_UNSUPPORTED, "experts %d > %d, topk %d > %d or groups %d > %d", experts,
                     AR_MAX_EXPERTS, topk, AR_MAX_TOPK, groups, AR_MAX_GROUPS);
    if (experts % groups != 0)
        return efail(AR_ERR_INVALID, "groups %d does not divide experts %d", groups, experts);
    if (groups_kept < 1 || groups_kept > groups)
        return efail(AR_ERR_INVALID, "groups_kept %d outside 1..%d", groups_kept, groups);
    if (topk > groups_kept * (experts / groups))
        return efail(AR_ERR_INVALID, "topk %d > the %d experts of %d groups", topk,
                     groups_kept * (experts / groups), groups_kept);
    if (score != AR_SCORE_SOFTMAX && score != AR_SCORE_SIGMOID)
        return efail(AR_ERR_INVALID, "score %d unknown", score);
    if (group_score != AR_GROUP_MAX && group_score != AR_GROUP_TOP2)
        return efail(AR_ERR_INVALID, "group_score %d unknown", group_score);
    if (renormalize != 0 && renormalize != 1)
        return efail(AR_ERR_INVALID, "renormalize %d is not 0 or 1", renormalize);
    if (tokens == 0)
        return AR_OK;
    if (!aligned(logits, 16))
        return efail(AR_ERR_INVALID, "logits NULL or not 16-byte aligned");
    if (((uintptr_t)bias & 3) || !aligned(ids_out, 4) || !aligned(weights_out, 4))
        return efail(AR_ERR_INVALID, "bias misaligned, or ids_out or weights_out NULL or misaligned");
    const RouteArgs a{logits, bias, tokens, experts, score, groups, groups_kept, group_score, topk,
                      renormalize, scale, ids_out, weights_out};
    return launched(launch_route(dtype, a, static_cast<cudaStream_t>(stream)), "route kernel launch");
}

int ar_fusion_expert_plan(const int32_t* ids, int tokens, int topk, int first_expert,
                          int experts, int32_t* offsets_out, int32_t* position_out,
                          void* stream)
{
    if (tokens < 0 || topk < 1 || first_expert < 0 || experts < 1)
        return efail(AR_ERR_INVALID, "tokens %d or first_expert %d < 0, topk %d or experts %d < 1",
                     tokens, first_expert, topk, experts);
    if (experts > AR_MAX_EXPERTS)
        return efail(AR_ERR_UNSUPPORTED, "experts %d > %d", experts, AR_MAX_EXPERTS);
    if ((long long)tokens * topk > INT_MAX || first_expert > INT_MAX - experts)
        return efail(AR_ERR_UNSUPPORTED, "tokens %d x topk %d or first_expert %d beyond 2^31 - 1",
                     tokens, topk, first_expert);
    if (!aligned(offsets_out, 4))
        return efail(AR_ERR_INVALID, "offsets_out NULL or misaligned");
    if (tokens > 0 && (!aligned(ids, 4) || !aligned(position_out, 4)))
        return efail(AR_ERR_INVALID, "ids or position_out NULL or misaligned");
    const PlanArgs a{ids, tokens * topk, first_expert, experts, offsets_out, position_out};
    return launched(launch_plan(a, static_cast<cudaStream_t>(stream)), "plan kernel launch");
}

int ar_fusion_quant_blocks(const void* in, int rows, int hidden, int dtype, int activation,
                           const int32_t* position, int copies, const int32_t* row_count,
                           int out_rows, void* quant_out, float* scale_out, void* stream)
{
    if (!dtype_supported(dtype))
        return bad_dtype(dtype);
    if (rows < 0 || out_rows < 0)
        return efail(AR_ERR_INVALID, "rows %d or out_rows %d < 0", rows, out_rows);
    if (hidden < 16 || hidden % 16 != 0)
        return efail(AR_ERR_INVALID, "hidden %d is not a positive multiple of 16", hidden);
    if (hidden > kMaxLength)
        return efail(AR_ERR_UNSUPPORTED, "hidden %d > %d", hidden, kMaxLength);
    if (activation != AR_ACT_NONE && activation != AR_ACT_SILU_MUL)
        return efail(AR_ERR_INVALID, "activation %d unknown", activation);
    if (copies < 1 || (!position && copies != 1))
        return efail(AR_ERR_INVALID, "copies %d < 1, or not 1 without position", copies);
    if (!position && out_rows < rows)
        return efail(AR_ERR_INVALID, "out_rows %d < rows %d", out_rows, rows);
    if (rows == 0 || out_rows == 0)     // out_rows 0: every position lies outside
        return AR_OK;
    if (!aligned(in, 16) || !aligned(quant_out, 16))
        return efail(AR_ERR_INVALID, "in or quant_out NULL or not 16-byte aligned");
    if (!aligned(scale_out, 4) || ((uintptr_t)position & 3) || ((uintptr_t)row_count & 3))
        return efail(AR_ERR_INVALID, "scale_out NULL, or scale_out, position or row_count misaligned");
    const BlockQuantArgs a{static_cast<const uint8_t*>(in), rows, hidden, activation, position,
                           copies, row_count, out_rows, static_cast<uint8_t*>(quant_out), scale_out};
    return launched(launch_block_quant(dtype, a, static_cast<cudaStream_t>(stream)),
                    "block quantiser launch");
}

int ar_fusion_matmul_fp8(const void* a, const float* a_scale, const void* b,
                         const float* b_scale, int rows, int cols, int depth, int dtype,
                         void* out, void* stream)
{
    const MatmulArgs m{static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(b),
                       b_scale, nullptr, 1, rows, cols, depth, out};
    const int rc = check_matmul(m, dtype);
    if (rc || rows == 0)
        return rc;
    return launched(launch_matmul(dtype, m, static_cast<cudaStream_t>(stream)),
                    "matmul kernel launch");
}

int ar_fusion_expert_matmul_fp8(const void* a, const float* a_scale, const void* b,
                                const float* b_scale, const int32_t* offsets, int experts,
                                int rows, int cols, int depth, int dtype, void* out,
                                void* stream)
{
    const MatmulArgs m{static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(b),
                       b_scale, offsets, experts, rows, cols, depth, out};
    const int rc = check_matmul(m, dtype);
    if (rc)
        return rc;
    if (rows > 0 && !aligned(offsets, 4))
        return efail(AR_ERR_INVALID, "offsets NULL or misaligned");
    if (rows == 0)
        return AR_OK;
    return launched(launch_matmul(dtype, m, static_cast<cudaStream_t>(stream)),
                    "expert matmul kernel launch");
}

int ar_fusion_combine(const void* rows_in, int in_rows, const int32_t* position,
                      const float* weights, int tokens, int topk, int hidden, int dtype,
                      const void* add, void* out, void* stream)
{
    if (!dtype_supported(dtype))
        return bad_dtype(dtype);
    if (in_rows < 0 || tokens < 0 || topk < 1)
        return efail(AR_ERR_INVALID, "in_rows %d or tokens %d < 0, or topk %d < 1", in_rows, tokens,
                     topk);
    if (hidden < 8 || hidden % 8 != 0)
        return efail(AR_ERR_INVALID, "hidden %d is not a positive multiple of 8", hidden);
    if (tokens == 0)
        return AR_OK;
    if ((in_rows > 0 && !aligned(rows_in, 16)) || ((uintptr_t)add & 15) || !aligned(out, 16))
        return efail(AR_ERR_INVALID, "rows_in or out NULL or not 16-byte aligned, or add misaligned");
    if (!aligned(position, 4) || !aligned(weights, 4))
        return efail(AR_ERR_INVALID, "position or weights NULL or misaligned");
    const CombineArgs a{static_cast<const uint8_t*>(rows_in), in_rows, position, weights, tokens,
                        topk, hidden, static_cast<const uint8_t*>(add), static_cast<uint8_t*>(out)};
    return launched(launch_combine(dtype, a, static_cast<cudaStream_t>(stream)),
                    "combine kernel launch");
}

}  // extern "C"

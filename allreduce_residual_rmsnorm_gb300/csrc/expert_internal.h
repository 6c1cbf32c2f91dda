// Launchers behind the expert-layer entry points (not part of the C ABI).
// Each returns the cudaError_t of its launch; arguments are already checked.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ar_fusion.h"

namespace arf {

struct RouteArgs {
    const void* logits;         // [T][E] of dtype
    const float* bias;          // [E] or NULL
    int T, E, score, G, keep, group_score, k, renorm;
    float scale;
    int32_t* ids;               // [T][k]
    float* weights;             // [T][k]
};
cudaError_t launch_route(int dtype, const RouteArgs& a, cudaStream_t s);

struct PlanArgs {
    const int32_t* ids;         // [slots]
    int slots, first, E;
    int32_t* offsets;           // [E + 1]
    int32_t* position;          // [slots]
};
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s);

struct BlockQuantArgs {
    const uint8_t* in;
    int rows, hidden, act;
    const int32_t* position;    // [rows][copies] or NULL
    int copies;
    const int32_t* row_count;   // device scalar or NULL
    int out_rows;
    uint8_t* q;
    float* scale;
};
cudaError_t launch_block_quant(int dtype, const BlockQuantArgs& a, cudaStream_t s);

struct MatmulArgs {
    const uint8_t* a;           // [rows][depth] E4M3
    const float* sa;            // [rows][blocks]
    const uint8_t* b;           // [experts][cols][depth] E4M3
    const float* sb;            // [experts][ceil(cols / 128)][blocks]
    const int32_t* offsets;     // [experts + 1], NULL: one expert with every row
    int experts, rows, cols, depth;
    void* out;                  // [rows][cols]
};
cudaError_t launch_matmul(int dtype, const MatmulArgs& a, cudaStream_t s);

struct CombineArgs {
    const uint8_t* rows;
    int in_rows;
    const int32_t* position;    // [T][k]
    const float* weights;       // [T][k]
    int T, k, H;
    const uint8_t* add;         // [T][H] or NULL
    uint8_t* out;               // [T][H]
};
cudaError_t launch_combine(int dtype, const CombineArgs& a, cudaStream_t s);

// Launch with programmatic dependent launch: the blocks may be scheduled while
// the kernel before them on the stream finishes, and wait on the device
// (griddepcontrol.wait) before their first access to global memory.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Runs `set` the first time on each device (below 64; on others every time): the
// attributes of a kernel that outlast the call.  Two threads may both run it.
template <class F>
cudaError_t once_per_device(std::atomic<uint64_t>& done, F&& set)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    e = set();
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

inline int quant_blocks(int depth) { return (depth + AR_QUANT_BLOCK - 1) / AR_QUANT_BLOCK; }

}  // namespace arf

// Row layout sorted by expert: a stable counting sort of the slots in one
// launch of one cluster, without a workspace and without atomics whose order
// could show.  Each warp owns a run of consecutive slots and counts it by
// expert in shared memory; the counts are summed over the warps of a block
// and, through distributed shared memory, over the blocks of the cluster; the
// second pass over the same slots (an L2 hit) numbers them.
#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t ld_dsmem_u32(const void* local, unsigned rank)
{
    const uint32_t la = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(la), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

// shared memory: count[kWarps][E], total[E]
__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a)
{
    extern __shared__ uint32_t sh[];
    __shared__ uint32_t warp_sum[kWarps];
    const int E = a.E;
    uint32_t* total = sh + kWarps * E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* count = sh + warp * E;
    const unsigned blocks = cluster_size(), me = cluster_rank();

    // this warp's run of slots, whole rounds of 32 but for the last
    const int64_t rounds = ((int64_t)a.slots + 31) / 32;
    const int64_t warps = (int64_t)blocks * kWarps, w = (int64_t)me * kWarps + warp;
    const int64_t lo = rounds * w / warps * 32;
    const int64_t hi0 = rounds * (w + 1) / warps * 32;
    const int64_t hi = hi0 < a.slots ? hi0 : a.slots;

    for (int e = lane; e < E; e += 32)
        count[e] = 0;
    __syncwarp();
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const uint32_t e = (uint32_t)a.ids[i] - (uint32_t)a.first;
        if (e < (uint32_t)E)
            atomicAdd(&count[e], 1u);
    }
    __syncthreads();
    // counts of the warps before, per expert
    if (tid < E) {
        uint32_t run = 0;
        for (int v = 0; v < kWarps; ++v) {
            const uint32_t c = sh[v * E + tid];
            sh[v * E + tid] = run;
            run += c;
        }
        total[tid] = run;
    }
    cluster_barrier();
    uint32_t all = 0, before = 0;
    if (tid < E) {
        for (unsigned b = 0; b < blocks; ++b) {
            const uint32_t c = ld_dsmem_u32(&total[tid], b);
            before += b < me ? c : 0u;
            all += c;
        }
    }
    // exclusive sum over experts (threads)
    uint32_t inc = all;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, m);
        inc += lane >= m ? v : 0u;
    }
    if (lane == 31)
        warp_sum[warp] = inc;
    cluster_barrier();          // every total has been read
    uint32_t first = inc - all;
    for (int v = 0; v < warp; ++v)
        first += warp_sum[v];
    if (tid < E) {
        total[tid] = first + before;
        if (me == 0) {
            a.offsets[tid] = (int32_t)first;
            if (tid == E - 1)
                a.offsets[E] = (int32_t)(first + all);
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const uint32_t e = i < hi ? (uint32_t)a.ids[i] - (uint32_t)a.first : 0xffffffffu;
        const bool local = e < (uint32_t)E;
        const uint32_t same = __match_any_sync(0xffffffffu, local ? e : 0xffffffffu);
        const uint32_t earlier = __popc(same & ((1u << lane) - 1u));
        const uint32_t base = local ? total[e] + count[e] : 0u;
        if (i < hi)
            a.position[i] = local ? (int32_t)(base + earlier) : -1;
        __syncwarp();
        if (local && earlier == 0)
            count[e] += __popc(same);
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s)
{
    const size_t smem = sizeof(uint32_t) * (size_t)(kWarps + 1) * a.E;
    cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(uint32_t) * (kWarps + 1) * AR_MAX_EXPERTS));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    const unsigned blocks = a.slots <= 4 * kThreads ? 1 : 8;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

}  // namespace arf

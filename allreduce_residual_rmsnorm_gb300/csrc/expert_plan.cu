// Row layout sorted by expert: a stable counting sort of the slots in one
// launch of one cluster, without a workspace and without atomics whose order
// could show.  Each warp owns a run of consecutive slots and counts it by
// expert in shared memory; the counts are summed over the warps of a block
// and, through distributed shared memory, over the blocks of the cluster; the
// second pass over the same slots (a cache hit) numbers them.
//
// Bounded by latency: the ids are 256 KB at 8192 tokens of 8 experts.  So the
// loads of 8 rounds are in flight at once, and small calls take few warps.
#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kRounds = 8;      // of 32 slots, loaded together
constexpr int kPerThread = 4;   // experts of a thread at most: blocks have 256 threads or more
constexpr int kBlocks = 8;      // of the cluster, or as many as one may have
constexpr int kMaxBlocks = 16;

__device__ __forceinline__ uint32_t ld_dsmem_u32(const void* local, unsigned rank)
{
    const uint32_t la = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(la), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

// The local experts of the slots of 8 rounds (~0 for a slot of none), and the
// lanes of each round with the same one.  The latter by one ballot per bit of
// the expert's number: a few instructions of full rate each, where one
// match.any took 8192 tokens of 8 experts 13 us in all.
__device__ __forceinline__ void load_rounds(const PlanArgs& a, int bits, int64_t i, int64_t hi,
                                            uint32_t (&e)[kRounds], uint32_t (&same)[kRounds])
{
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        e[r] = i + 32 * r < hi ? (uint32_t)a.ids[i + 32 * r] : 0xffffffffu;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t local = e[r] - (uint32_t)a.first;
        const bool in = i + 32 * r < hi && local < (uint32_t)a.E;
        e[r] = in ? local : 0xffffffffu;
        same[r] = __ballot_sync(0xffffffffu, in);
    }
    for (int k = 0; k < bits; ++k) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint32_t ones = __ballot_sync(0xffffffffu, e[r] >> k & 1u);
            same[r] &= e[r] >> k & 1u ? ones : ~ones;
        }
    }
}

// shared memory: count[warps][E], total[E]
__global__ void __launch_bounds__(32 * kMaxWarps) plan_kernel(PlanArgs a, int bits)
{
    extern __shared__ uint32_t sh[];
    __shared__ uint32_t warp_sum[kMaxWarps];
    const int E = a.E;
    const int threads = blockDim.x, warps = threads / 32;
    uint32_t* total = sh + warps * E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* count = sh + warp * E;
    const unsigned blocks = cluster_size(), me = cluster_rank();

    // this warp's run of slots, whole rounds of 32 but for the last
    const int64_t rounds = ((int64_t)a.slots + 31) / 32;
    const int64_t all_warps = (int64_t)blocks * warps, w = (int64_t)me * warps + warp;
    const int64_t lo = rounds * w / all_warps * 32;
    const int64_t hi0 = rounds * (w + 1) / all_warps * 32;
    const int64_t hi = hi0 < a.slots ? hi0 : a.slots;

    pdl_trigger();
    for (int e = lane; e < E; e += 32)
        count[e] = 0;
    pdl_wait();
    const uint32_t below = (1u << lane) - 1u;
    uint32_t e[kRounds], same[kRounds];
    load_rounds(a, bits, lo + lane, hi, e, same);
    __syncwarp();
    for (int64_t i = lo;;) {
        // the first lane of each expert adds for all: no two lanes of a warp
        // touch the same counter
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (e[r] != 0xffffffffu && (same[r] & below) == 0)
                atomicAdd(&count[e[r]], (uint32_t)__popc(same[r]));
        i += 32 * kRounds;
        if (i >= hi)
            break;
        load_rounds(a, bits, i + lane, hi, e, same);
    }
    __syncthreads();
    // counts of the warps before, per expert
    for (int x = tid; x < E; x += threads) {
        uint32_t run = 0;
#pragma unroll 8
        for (int v = 0; v < warps; ++v) {
            const uint32_t c = sh[v * E + x];
            sh[v * E + x] = run;
            run += c;
        }
        total[x] = run;
    }
    if (blocks > 1)
        cluster_barrier();
    else
        __syncthreads();
    // consecutive experts of a thread: their rows in the cluster, and in the
    // blocks before this one
    const int per = (E + threads - 1) / threads;
    uint32_t all[kPerThread], before[kPerThread], mine = 0;
#pragma unroll
    for (int q = 0; q < kPerThread; ++q) {
        const int x = tid * per + q;
        all[q] = before[q] = 0;
        if (q < per && x < E) {
            if (blocks > 1) {
                uint32_t c[kMaxBlocks];         // every block's at once
#pragma unroll
                for (unsigned b = 0; b < kMaxBlocks; ++b)
                    c[b] = b < blocks ? ld_dsmem_u32(&total[x], b) : 0u;
#pragma unroll
                for (unsigned b = 0; b < kMaxBlocks; ++b) {
                    before[q] += b < me ? c[b] : 0u;
                    all[q] += c[b];
                }
            } else {
                all[q] = total[x];
            }
        }
        mine += all[q];
    }
    // exclusive sum over threads
    uint32_t inc = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, m);
        inc += lane >= m ? v : 0u;
    }
    if (lane == 31)
        warp_sum[warp] = inc;
    if (blocks > 1)
        cluster_barrier();      // every total has been read
    else
        __syncthreads();
    uint32_t first = inc - mine;
    // sums of the warps before
    uint32_t part = lane < warp ? warp_sum[lane] : 0u;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        part += __shfl_xor_sync(0xffffffffu, part, m);
    first += part;
#pragma unroll
    for (int q = 0; q < kPerThread; ++q) {
        const int x = tid * per + q;
        if (q < per && x < E) {
            total[x] = first + before[q];
            if (me == 0) {
                a.offsets[x] = (int32_t)first;
                if (x == E - 1)
                    a.offsets[E] = (int32_t)(first + all[q]);
            }
            first += all[q];
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kRounds) {
        if (hi - lo > 32 * kRounds)     // else they are still in registers
            load_rounds(a, bits, i0 + lane, hi, e, same);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t i = i0 + 32 * r + lane;
            if (i0 + 32 * r >= hi)
                break;
            const bool local = e[r] != 0xffffffffu;
            const uint32_t earlier = __popc(same[r] & below);
            const uint32_t base = local ? total[e[r]] + count[e[r]] : 0u;
            if (i < hi)
                a.position[i] = local ? (int32_t)(base + earlier) : -1;
            __syncwarp();
            if (local && earlier == 0)
                count[e[r]] += __popc(same[r]);
            __syncwarp();
        }
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s)
{
    // devices where a cluster of 16 blocks fits
    static std::atomic<uint64_t> done{0}, sixteen{0};
    const int most = (int)(sizeof(uint32_t) * (kMaxWarps + 1) * AR_MAX_EXPERTS);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = once_per_device(done, [&] {
            const cudaError_t es = cudaFuncSetAttribute(
                plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            if (es != cudaSuccess || dev >= 64)
                return es;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kMaxBlocks);
            cfg.blockDim = dim3(32 * kMaxWarps);
            cfg.dynamicSmemBytes = most;
            cudaLaunchAttribute at;
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = kMaxBlocks;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            int fit = 0;
            if (cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                     1) == cudaSuccess &&
                cudaOccupancyMaxActiveClusters(&fit, plan_kernel, &cfg) == cudaSuccess && fit > 0)
                sixteen.fetch_or(1ull << dev);
            else
                (void)cudaGetLastError();       // 8 blocks then
            return cudaSuccess;
        });
    if (e != cudaSuccess)
        return e;
    // One block up to four rounds a warp, 8 up to six, then 16 (8 against 16, with
    // the routing before: 32768 slots 17.1 / 17.4 us, 65536 25.3 / 24.8, 131072,
    // where 8 would load their rounds twice, 48.0 / 38.6).  8 warps at least, for
    // the experts.
    const int64_t rounds = ((int64_t)a.slots + 31) / 32;
    const bool many = rounds > 6 * kBlocks * kMaxWarps && dev < 64 &&
                      (sixteen.load(std::memory_order_acquire) >> dev & 1u);
    const unsigned blocks = rounds <= 4 * kMaxWarps ? 1 : many ? kMaxBlocks : kBlocks;
    const int warps = rounds <= 8 ? 8 : rounds <= 16 ? 16 : kMaxWarps;
    static_assert(8 * 32 * kPerThread >= AR_MAX_EXPERTS, "experts of a block of 8 warps");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = sizeof(uint32_t) * (size_t)(warps + 1) * a.E;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    int bits = 0;               // of the largest local expert's number
    while ((1 << bits) < a.E)
        ++bits;
    return cudaLaunchKernelEx(&cfg, plan_kernel, a, bits);
}

}  // namespace arf

// 8-bit product for few rows per expert: the weights are read once and bound
// the time, so they take the 128 lanes of tensor memory (128 columns of the
// output per block) and the token rows its columns, 16 to 64 at a time.
//
// The depth is split over the blocks of a cluster where one block per 128
// columns would leave SMs idle; their fp32 sums meet in distributed shared
// memory, added in rank order by the block that stores them, so no workspace
// and no atomics are needed and the result does not depend on timing.
//
// Each block of 128 of the depth goes to a tensor-memory buffer of its own and
// is added, times sa * sb, to fp32 registers: a thread has one column of the
// output, the rows' scales come through shared memory, made ahead by two warps.
//
// Shared memory is sized so that at most two blocks share an SM (three where a
// block has 64 columns of tensor memory), which keeps their tensor memory (256
// columns each at most) within the SM's 512: no block of a cluster can wait for
// tensor memory that waits for its cluster.
//
// Weights that one block alone reads leave L2 first (16 rows: 28672 x 7168 33.3 ->
// 32.0 us, 131072 x 2048 48.5 -> 42.8); with several row tiles of an expert that
// cost 1%, and where all of them may stay in L2 for a next call it cost 13% of
// that (1 x 7168 x 2048, 14.7 MB), so there they are left alone.
//
// Warps 0-3: add and store; warp 4: copies; warp 5: products; warps 6, 7: scales.
#include "matmul_internal.h"
#include "tensor_core.cuh"

namespace arf {
namespace {

constexpr int kN = 128, kK = 128;          // columns per block, depth per step
constexpr int kBytesW = kN * kK;
constexpr int kThreads = 256;
constexpr int kMaxStages = 10, kMaxSplit = 8;
constexpr int kBufs = 4;                   // of tensor memory
constexpr int kAhead = 8;                  // blocks of the depth per group of scales

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

__device__ __forceinline__ float ld_dsmem_f32(const float* local, unsigned rank)
{
    uint32_t ra;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
}

template <class D, int TOK>
__global__ void __launch_bounds__(kThreads)
    matmul_narrow_kernel(const __grid_constant__ CUtensorMap map_a,
                         const __grid_constant__ CUtensorMap map_b, MatmulArgs a, int* status,
                         int split, int stages, int large)
{
    constexpr uint32_t kCols = TOK * kBufs;
    constexpr int kStage = kBytesW + TOK * kK;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(16) float scale_sh[2][kAhead][TOK];     // two groups of scales
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2 * kBufs + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int e = blockIdx.z;
    pdl_trigger();
    int row0 = 0, row1 = a.rows;
    if (a.offsets) {
        pdl_wait();
        row0 = min(max(a.offsets[e], 0), a.rows);
        row1 = min(max(a.offsets[e + 1], row0), a.rows);
    }
    // the same for every block of the cluster: all leave, or none
    if (row0 + (int64_t)blockIdx.y * TOK >= row1)
        return;

    const uint32_t stage0 = (smem_u32(dyn) + 1023u) & ~1023u;
    float* sums = reinterpret_cast<float*>(dyn + (stage0 - smem_u32(dyn)) + stages * kStage);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxStages,
                   tfull = empty + 8 * kMaxStages, tempty = tfull + 8 * kBufs,
                   sfull = tempty + 8 * kBufs, sempty = sfull + 16, done = sempty + 16;
    const Bail bail{smem_u32(&dead), status};
    if (tid == 0) {
        dead = 0;
        for (int s = 0; s < stages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            bar_init(tfull + 8 * b, 1);
            bar_init(tempty + 8 * b, 4);
        }
        for (int g = 0; g < 2; ++g) {
            bar_init(sfull + 8 * g, 2);
            bar_init(sempty + 8 * g, 4);
        }
        bar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
    }
    if (warp == 5)
        tmem_alloc(smem_u32(&tmem_slot), kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    const int rank = blockIdx.x % split;
    const int n0 = blockIdx.x / split * kN;
    const int nkb = (a.depth + kK - 1) / kK;
    const int kb0 = (int)((int64_t)nkb * rank / split), kb1 = (int)((int64_t)nkb * (rank + 1) / split);
    const int64_t step = (int64_t)gridDim.y * TOK;

    // per role: position in the ring of stages and of tensor-memory buffers
    uint32_t s = 0, ph = 0, it = 0, grp = 0, issued = 0;
    bool ok = true;
    for (int64_t m0 = row0 + (int64_t)blockIdx.y * TOK; m0 < row1; m0 += step) {
        if (warp == 4) {
            const int brow = e * a.cols + n0;
            const uint64_t policy = large && row1 - row0 <= TOK ? evict_first() : evict_normal();
            for (int kb = kb0; kb < kb1 && ok; ++kb) {
                ok = __all_sync(0xffffffffu, bar_wait(empty + 8 * s, ph ^ 1, bail, 1));
                if (!ok)
                    break;
                if (elect_one()) {
                    const uint32_t at = stage0 + s * kStage;
                    bar_expect(full + 8 * s, kStage);
                    tma_load_2d(at, &map_b, full + 8 * s, kb * kK, brow, policy);
                    tma_load_2d(at + kBytesW, &map_a, full + 8 * s, kb * kK, (int)m0);
                }
                __syncwarp();
                ++issued;
                if (++s == (uint32_t)stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        } else if (warp == 5) {
            if (elect_one()) {
                constexpr uint32_t idesc = fp8_idesc(kN, TOK);
                const uint64_t desc0 = smem_desc(stage0);
                for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
                    const uint32_t b = it % kBufs;
                    if (!(ok = bar_wait(full + 8 * s, ph, bail, 3)) ||
                        !(ok = bar_wait(tempty + 8 * b, (it / kBufs & 1) ^ 1, bail, 2)))
                        break;
                    tc_fence_after();
                    const uint32_t w = (uint32_t)desc0 + s * (kStage >> 4);
                    mma4_fp8(tmem + b * TOK, w, w + (kBytesW >> 4), (uint32_t)(desc0 >> 32), idesc);
                    mma_commit(empty + 8 * s);
                    mma_commit(tfull + 8 * b);
                    if (++s == (uint32_t)stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            __syncwarp();
        } else if (warp >= 6) {
            // a group of blocks of the depth in flight per row
            const int have = (int)min((int64_t)TOK, row1 - m0);
            const int ncb = (a.cols + AR_QUANT_BLOCK - 1) / AR_QUANT_BLOCK;
            const float* sb = a.sb + ((uint64_t)e * ncb + n0 / AR_QUANT_BLOCK) * nkb;
            for (int kb = kb0; kb < kb1 && ok; kb += kAhead, ++grp) {
                const uint32_t g = grp & 1;
                float v[kAhead];
                const int r = 32 * (warp - 6) + lane;
                const float* sa = a.sa + (uint64_t)(m0 + (r < have ? r : 0)) * nkb;
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int k = min(kb + j, kb1 - 1);
                    const float f = sb[k];
                    v[j] = r < TOK ? sa[k] * f : 0.0f;
                }
                ok = __all_sync(0xffffffffu, bar_wait(sempty + 8 * g, (grp >> 1 & 1) ^ 1, bail, 5));
                if (!ok)
                    break;
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    if (r < TOK)
                        scale_sh[g][j][r] = v[j];
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(sfull + 8 * g);
            }
        } else {
            // A wait that gives up is not looked at here: the sums are then
            // undefined as the status says, and every later wait returns at once.
            const int have = (int)min((int64_t)TOK, row1 - m0);
            const int n = n0 + tid;
            uint64_t acc[TOK / 2];
#pragma unroll
            for (int i = 0; i < TOK / 2; ++i)
                acc[i] = 0ull;
            for (int kg = kb0; kg < kb1; kg += kAhead, ++grp) {
                const uint32_t g = grp & 1;
                bar_wait(sfull + 8 * g, grp >> 1 & 1, bail, 6);
                const int steps = min(kAhead, kb1 - kg);
                for (int j = 0; j < steps; ++j, ++it) {
                    const uint32_t b = it % kBufs;
                    bar_wait(tfull + 8 * b, it / kBufs & 1, bail, 4);
                    __syncwarp();
                    tc_fence_after();
                    const float4* sc = reinterpret_cast<const float4*>(scale_sh[g][j]);
                    const uint32_t from = tmem + ((uint32_t)(32 * warp) << 16) + b * TOK;
                    uint32_t d[2][16];
                    tmem_ld16(from, d[0]);
#pragma unroll
                    for (int c = 0; c < TOK / 16; ++c) {
                        tmem_wait(d[c & 1]);
                        if (c + 1 < TOK / 16)
                            tmem_ld16(from + 16 * (c + 1), d[(c + 1) & 1]);
                        if (c + 1 == TOK / 16) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                bar_arrive(tempty + 8 * b);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 f = sc[4 * c + i];
                            fma_pair(acc[8 * c + 2 * i],
                                     pack_pair(d[c & 1][4 * i], d[c & 1][4 * i + 1]),
                                     pair_of(f.x, f.y));
                            fma_pair(acc[8 * c + 2 * i + 1],
                                     pack_pair(d[c & 1][4 * i + 2], d[c & 1][4 * i + 3]),
                                     pair_of(f.z, f.w));
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(sempty + 8 * g);
            }
            if (split == 1) {
                if (n < a.cols) {
#pragma unroll
                    for (int i = 0; i < TOK / 2; ++i) {
                        const float2 f = unpack_pair(acc[i]);
                        if (2 * i < have)
                            store1<D>(a.out, (uint64_t)(m0 + 2 * i) * a.cols + n, f.x);
                        if (2 * i + 1 < have)
                            store1<D>(a.out, (uint64_t)(m0 + 2 * i + 1) * a.cols + n, f.y);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < TOK / 2; ++i) {
                    const float2 f = unpack_pair(acc[i]);
                    sums[(2 * i) * kN + tid] = f.x;
                    sums[(2 * i + 1) * kN + tid] = f.y;
                }
            }
        }
        if (split > 1) {
            cluster_barrier();
            if (warp < 4) {
                const int have = (int)min((int64_t)TOK, row1 - m0);
                const int n = n0 + tid;
                // four of this block's rows from all blocks before the first
                // addition: one at a time their latency was most of a small call
                for (int c0 = rank; c0 < have; c0 += 4 * split) {
                    float part[4][kMaxSplit];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int q = 0; q < kMaxSplit; ++q)
                            if (q < split && c0 + i * split < have)
                                part[i][q] = ld_dsmem_f32(sums + (c0 + i * split) * kN + tid, q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = c0 + i * split;
                        float v = 0.0f;
#pragma unroll
                        for (int q = 0; q < kMaxSplit; ++q)
                            v += q < split && c < have ? part[i][q] : 0.0f;
                        if (c < have && n < a.cols)
                            store1<D>(a.out, (uint64_t)(m0 + c) * a.cols + n, v);
                    }
                }
            }
            cluster_barrier();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Without a wait that gave up every product has been added, so no copy and no
    // product is left.  With one, whichever warp's it was, both end here before
    // the block does.
    if (*static_cast<volatile int*>(&dead)) {
        if (warp == 4) {
            for (uint32_t i = 0; i < (uint32_t)stages && i < issued; ++i) {
                ph ^= s == 0;
                s = s == 0 ? stages - 1 : s - 1;
                bar_drain(full + 8 * s, ph);
            }
        } else if (warp == 5) {
            if (elect_one())
                mma_commit(done);
            __syncwarp();
            bar_drain(done, 0);
        }
    }
    if (warp == 5)
        tmem_free(tmem, kCols);
}

template <class D, int TOK>
cudaError_t launch_t(const MatmulArgs& a, int split, const DeviceInfo& d, cudaStream_t s)
{
    CUtensorMap map_a, map_b;
    if (!byte_tensor_map(&map_a, a.a, (uint64_t)a.rows, (uint64_t)a.depth, TOK) ||
        !byte_tensor_map(&map_b, a.b, (uint64_t)a.experts * a.cols, (uint64_t)a.depth, kN))
        return cudaErrorInvalidValue;
    constexpr int kStage = kBytesW + TOK * kK;
    const int64_t per = ((int64_t)a.rows + a.experts - 1) / a.experts;
    const int64_t y = (per + TOK - 1) / TOK;
    const int64_t x = (int64_t)((a.cols + kN - 1) / kN) * split;
    // Two blocks per SM; three of 16 rows (their registers allow it) where there
    // are six or more to an SM, so that more of a block's start and end passes
    // behind the others' copies: 64 experts x 4096 x 2048, 128 rows, 68.5 -> 65.3
    // us, x 2048 x 512 16.3 -> 13.2.  With fewer it is the stages that count: 512
    // blocks of 65536 x 2048 25.9 against 26.3 us.
    constexpr int kMost = 106 * 1024, kThird = 73 * 1024;
    const bool third = TOK == 16 && (a.experts < a.rows ? a.experts : a.rows) * x * y >= 6 * d.sms;
    const int smem = third ? kThird : kMost;    // the whole of it: never another block
    const int sums = split > 1 ? TOK * kN * 4 : 0;
    int stages = (smem - sums - 1024) / kStage;
    stages = stages > kMaxStages ? kMaxStages : stages;
    const auto kernel = matmul_narrow_kernel<D, TOK>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    });
    if (e != cudaSuccess)
        return e;
    // half of L2: beside what else a step touches, more would not stay
    const int large = (uint64_t)a.experts * a.cols * a.depth > 64ull << 20;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x, (unsigned)(y > 65535 ? 65535 : y), a.experts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, map_a, map_b, a, d.status, split, stages, large);
}

template <class D>
cudaError_t launch_d(const MatmulArgs& a, int tokens, int split, const DeviceInfo& d,
                     cudaStream_t s)
{
    switch (tokens) {
    case 16: return launch_t<D, 16>(a, split, d, s);
    case 32: return launch_t<D, 32>(a, split, d, s);
    default: return launch_t<D, 64>(a, split, d, s);
    }
}

}  // namespace

cudaError_t launch_matmul_narrow(int dtype, const MatmulArgs& a, int tokens, int split,
                                 const DeviceInfo& d, cudaStream_t s)
{
    switch (dtype) {
    case AR_DT_BF16: return launch_d<Bf16>(a, tokens, split, d, s);
    case AR_DT_FP16: return launch_d<Fp16>(a, tokens, split, d, s);
    default: return launch_d<F32>(a, tokens, split, d, s);
    }
}

}  // namespace arf

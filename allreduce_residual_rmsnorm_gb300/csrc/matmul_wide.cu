// 8-bit product for many rows: 128 rows x 256 columns of the output per tile,
// persistent blocks, one per SM.
//
// The scales change every 128 of the depth, so the tensor cores' sum of one
// block cannot stay in tensor memory: each block of 128 x 256 x 128 goes to one
// of two tensor-memory buffers, and 8 warps add it, times sa * sb, to fp32
// registers while the tensor cores fill the other buffer.  A row of the tile
// is a lane of tensor memory, so a thread has one row and one scale per block;
// its 128 columns are one scale block of the weights.
//
// Warps 0-7: add and store (warp w: rows 32 (w % 4), columns 128 (w / 4));
// warp 8: copies; warp 9: products.
#include "matmul_internal.h"
#include "tensor_core.cuh"

namespace arf {
namespace {

constexpr int kM = 128, kN = 256, kK = 128;
constexpr int kStages = 4;
constexpr int kBytesA = kM * kK, kBytesB = kN * kK, kStage = kBytesA + kBytesB;
constexpr int kThreads = 320;
constexpr int kSmem = kStages * kStage + 1024;      // 1024: alignment of the swizzle pattern
constexpr uint32_t kCols = 512;                     // tensor memory: two buffers of 256

struct Tile {
    int row, end, n, e;         // first row, end of the expert's rows, first column, expert
};

// Tiles are numbered expert by expert, within an expert in groups of 16 row
// tiles, rows fastest, so that blocks that run together share weights and rows.
__device__ __forceinline__ Tile tile_at(int64_t t, const int* first_tile, const int* first_row,
                                        int E, int ntn)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {       // the last expert whose tiles start at or before t
        const int mid = (lo + hi) >> 1;
        if ((int64_t)first_tile[mid] * ntn <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int mt = first_tile[lo + 1] - first_tile[lo];
    const int l = (int)(t - (int64_t)first_tile[lo] * ntn);
    const int group = l / (16 * ntn), in = l - group * 16 * ntn;
    const int tall = min(16, mt - group * 16);
    const int n = in / tall, m = group * 16 + in - n * tall;
    return Tile{first_row[lo] + m * kM, first_row[lo + 1], n * kN, lo};
}

// 16 consecutive columns of a row
template <class D>
__device__ __forceinline__ void store16(uint8_t* p, const uint64_t (&v)[8], int valid, int align)
{
    uint32_t w[16 * D::bytes / 4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack_pair(v[i]);
        if constexpr (D::bytes == 4) {
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
        } else {
            w[i] = pack2<D>(f.x, f.y);
        }
    }
    constexpr int kWords = 16 * D::bytes / 4;
    if (valid >= 16 && align >= 32) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + 4 * i),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                         "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                         : "memory");
    } else if (valid >= 16 && align >= 16) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < valid) {
                if constexpr (D::bytes == 4)
                    reinterpret_cast<uint32_t*>(p)[i] = w[i];
                else
                    reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

template <class D>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_wide_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, MatmulArgs a, int* status,
                       int align)
{
    extern __shared__ uint8_t dyn[];
    __shared__ int first_tile[AR_MAX_EXPERTS + 1], first_row[AR_MAX_EXPERTS + 1];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t stage0 = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages,
                   tempty = tfull + 16, done = tempty + 16;
    const Bail bail{&dead, status};

    if (tid == 0) {
        dead = 0;
        for (int s = 0; s < kStages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(tfull + 8 * b, 1);
            bar_init(tempty + 8 * b, 8);
        }
        bar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
    }
    if (warp == 9)
        tmem_alloc(smem_u32(&tmem_slot), kCols);
    // rows and row tiles before each expert
    if (warp == 0) {
        int tiles = 0, before = 0;
        for (int e0 = 0; e0 <= a.experts; e0 += 32) {
            const int e = e0 + lane;
            // clamped, and made not to decrease: every row has one expert at most
            int lo = e < a.experts ? 0 : a.rows;
            if (a.offsets && e <= a.experts)
                lo = min(max(a.offsets[e], 0), a.rows);
            lo = max(lo, before);
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, lo, m);
                lo = lane >= m ? max(lo, v) : lo;
            }
            if (e <= a.experts)
                first_row[e] = lo;
            before = __shfl_sync(0xffffffffu, lo, 31);
        }
        __syncwarp();
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane;
            const int t = e < a.experts ? (first_row[e + 1] - first_row[e] + kM - 1) / kM : 0;
            int inc = t;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, m);
                inc += lane >= m ? v : 0;
            }
            if (e < a.experts)
                first_tile[e] = tiles + inc - t;
            tiles += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0)
            first_tile[a.experts] = tiles;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int ntn = (a.cols + kN - 1) / kN;
    const int64_t tiles = (int64_t)first_tile[a.experts] * ntn;
    const int nkb = (a.depth + kK - 1) / kK;

    if (warp == 8) {
        if (lane == 0) {
            uint32_t s = 0, ph = 0, issued = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile x = tile_at(t, first_tile, first_row, a.experts, ntn);
                const int brow = x.e * a.cols + x.n;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!(ok = bar_wait(empty + 8 * s, ph ^ 1, bail, 1)))
                        break;
                    const uint32_t at = stage0 + s * kStage;
                    bar_expect(full + 8 * s, kStage);
                    tma_load_2d(at, &map_a, full + 8 * s, kb * kK, x.row);
                    tma_load_2d(at + kBytesA, &map_b, full + 8 * s, kb * kK, brow);
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // a block that gave up waits for its copies in flight
            for (uint32_t i = 0; !ok && i < kStages && i < issued; ++i) {
                ph ^= s == 0;
                s = s == 0 ? kStages - 1 : s - 1;
                bar_drain(full + 8 * s, ph);
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t idesc = fp8_idesc(kM, kN);
            uint32_t s = 0, ph = 0, it = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const uint32_t b = it & 1;
                    if (!(ok = bar_wait(tempty + 8 * b, ((it >> 1) & 1) ^ 1, bail, 2)) ||
                        !(ok = bar_wait(full + 8 * s, ph, bail, 3)))
                        break;
                    tc_fence_after();
                    const uint64_t da = smem_desc(stage0 + s * kStage);
                    const uint64_t db = smem_desc(stage0 + s * kStage + kBytesA);
#pragma unroll
                    for (int k = 0; k < kK / 32; ++k)
                        mma_fp8(tmem + b * kN, da + 2 * k, db + 2 * k, idesc, k > 0);
                    mma_commit(empty + 8 * s);
                    mma_commit(tfull + 8 * b);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) {
                mma_commit(done);
                bar_drain(done, 0);
            }
        }
    } else {
        const int half = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * 128;
        uint32_t it = 0;
        bool ok = true;
        const int ncb = (a.cols + AR_QUANT_BLOCK - 1) / AR_QUANT_BLOCK;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile x = tile_at(t, first_tile, first_row, a.experts, ntn);
            const int row = x.row + 32 * (warp & 3) + lane;
            const int n0 = x.n + 128 * half;
            const bool live = row < x.end && n0 < a.cols;
            const float* sa = a.sa + (uint64_t)(live ? row : 0) * nkb;
            const float* sb = a.sb + ((uint64_t)x.e * ncb + (n0 < a.cols ? n0 / AR_QUANT_BLOCK : 0)) * nkb;
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i)
                acc[i] = 0ull;
            float next = sa[0] * sb[0];
            for (int kb = 0; kb < nkb; ++kb, ++it) {
                const float sc = next;
                if (kb + 1 < nkb)
                    next = sa[kb + 1] * sb[kb + 1];
                const uint64_t s2 = pack_pair(__float_as_uint(sc), __float_as_uint(sc));
                const uint32_t b = it & 1;
                ok = __all_sync(0xffffffffu, bar_wait(tfull + 8 * b, (it >> 1) & 1, bail, 4));
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t from = lanes + b * kN;
                uint32_t d[2][16];
                tmem_ld16(from, d[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_wait(d[c & 1]);
                    if (c < 7)
                        tmem_ld16(from + 16 * (c + 1), d[(c + 1) & 1]);
                    if (c == 7) {
                        // everything of this buffer is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            bar_arrive(tempty + 8 * b);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        fma_pair(acc[8 * c + i], pack_pair(d[c & 1][2 * i], d[c & 1][2 * i + 1]), s2);
                }
            }
            if (ok && live) {
                uint8_t* p = static_cast<uint8_t*>(a.out) + ((uint64_t)row * a.cols + n0) * D::bytes;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint64_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = acc[8 * c + i];
                    store16<D>(p + 16 * c * D::bytes, v, a.cols - n0 - 16 * c, align);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9)
        tmem_free(tmem, kCols);
}

template <class D>
cudaError_t launch_t(const MatmulArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    CUtensorMap map_a, map_b;
    if (!byte_tensor_map(&map_a, a.a, (uint64_t)a.rows, (uint64_t)a.depth, kM) ||
        !byte_tensor_map(&map_b, a.b, (uint64_t)a.experts * a.cols, (uint64_t)a.depth, kN))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(matmul_wide_kernel<D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
        return e;
    // at most this many tiles: every expert may end in a part of one
    const int64_t most = ((int64_t)a.rows / kM + (a.experts < a.rows ? a.experts : a.rows)) *
                         ((a.cols + kN - 1) / kN);
    const unsigned grid = most < d.sms ? (unsigned)most : (unsigned)d.sms;
    const uint64_t where = (uint64_t)a.out | ((uint64_t)a.cols * D::bytes);
    const int align = where % 32 == 0 ? 32 : where % 16 == 0 ? 16 : 1;
    matmul_wide_kernel<D><<<grid, kThreads, kSmem, s>>>(map_a, map_b, a, d.status, align);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_matmul_wide(int dtype, const MatmulArgs& a, const DeviceInfo& d,
                               cudaStream_t s)
{
    switch (dtype) {
    case AR_DT_BF16: return launch_t<Bf16>(a, d, s);
    case AR_DT_FP16: return launch_t<Fp16>(a, d, s);
    default: return launch_t<F32>(a, d, s);
    }
}

}  // namespace arf

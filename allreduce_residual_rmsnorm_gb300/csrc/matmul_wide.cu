// 8-bit product for many rows: 256 rows x 256 columns of the output per tile
// and pair of blocks, persistent, one block per SM.
//
// The scales change every 128 of the depth, so the tensor cores' sum of one
// block of 128 cannot stay in tensor memory: each half of it (128 columns) goes
// to one of two buffers, and 4 warps add it, times sa * sb, to fp32 registers
// while the tensor cores fill the others.  A row of the tile is a lane of
// tensor memory, so a thread has one row and one scale per block; its 128
// columns are one scale block of the weights.  Halves, because the round trip
// of a buffer (products, commit, addition, release by both blocks: about 1400
// cycles) bounds the pair: with two buffers of 256 columns it was 935 cycles a
// block.
//
// A pair (cta_group::2) because the copies from L2 bound a block on its own:
// 128 x 256 needs 48 KB per 128 of the depth, and an SM took 53 bytes a cycle,
// 930 cycles for 512 of products.  In a pair each block brings its 128 rows and
// half the columns, 32 KB, and the tensor cores read the other half from the
// neighbour's shared memory.
//
// Warps 0-7: add and store (warp w: rows 32 (w % 4), columns 128 (w / 4));
// warp 8: copies; warp 9: products (of the pair's first block); warps 10, 11:
// the products of the scales, ahead of their use.
#include "ar_internal.h"
#include "matmul_internal.h"
#include "tensor_core.cuh"

namespace arf {
namespace {

constexpr int kM = 256, kN = 256, kK = 128;         // of a pair
constexpr int kHalf = 128;                          // rows, and columns of b, of one block
constexpr int kStages = 5;
constexpr int kBytes = kHalf * kK, kStage = 2 * kBytes;
constexpr int kThreads = 384;
// registers: launched with 168 each (65,536 / 384, in eights); the four warps
// that copy and issue give up what the eight that add take
constexpr int kRegsLaunch = 168, kRegsIssue = 88, kRegsAdd = 208;
static_assert(4 * kRegsIssue + 8 * kRegsAdd <= 12 * kRegsLaunch, "register shares");
constexpr int kOutRow = 64, kOutBuf = 32 * kOutRow;  // a store of 32 rows x 64 bytes
constexpr int kOutBufs = 2;                          // per adding warp
constexpr int kSmemOut = 8 * kOutBufs * kOutBuf;
constexpr int kSmem = kStages * kStage + kSmemOut + 1024;   // 1024: alignment of the swizzle
constexpr uint32_t kCols = 512;                     // tensor memory: four buffers of 128
constexpr int kAhead = 8;                           // blocks of the depth per group of scales

struct Tile {
    int row, end, n, e;         // first row, end of the expert's rows, first column, expert
};

// Tiles are numbered expert by expert, within an expert in groups of 8 row
// tiles, rows fastest, so that pairs that run together share weights and rows.
__device__ __forceinline__ Tile tile_at(int t, const int* first_tile, const int* first_row, int E,
                                        int ntn)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {       // the last expert whose tiles start at or before t
        const int mid = (lo + hi) >> 1;
        if (first_tile[mid] * ntn <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int mt = first_tile[lo + 1] - first_tile[lo];
    const int l = t - first_tile[lo] * ntn;
    const int group = l / (8 * ntn), in = l - group * 8 * ntn;
    const int tall = min(8, mt - group * 8);
    const int n = in / tall, m = group * 8 + in - n * tall;
    return Tile{first_row[lo] + m * kM, first_row[lo + 1], n * kN, lo};
}

// 16 consecutive columns of a row as words of the output type
template <class D>
__device__ __forceinline__ void round16(const uint64_t (&v)[8], uint32_t (&w)[16 * D::bytes / 4])
{
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
}

// the same stored directly: the rows of a tile that other rows follow
template <class D>
__device__ __forceinline__ void store16(uint8_t* p, const uint32_t (&w)[16 * D::bytes / 4],
                                        int valid, bool wide)
{
    if (valid >= 16 && wide) {
#pragma unroll
        for (int i = 0; i < 16 * D::bytes / 4; i += 4)
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

// Waits for what a pair that gave up has in flight; one warp of each block, none
// of which issues anything any more.  The copies of both blocks arrive at the
// first one's `full`: a stage is filled again only after the products of its last
// fill, so the blocks differ by one fill of a stage at most, of which the first
// block armed the barrier for both or not at all.  The commits arrive at the
// barriers of both.
__device__ __noinline__ void end_pair(uint32_t rank, uint32_t full, uint32_t empty, uint32_t tfull,
                                      const uint32_t* issued, const uint32_t* committed)
{
    const auto fills = [](uint32_t n, uint32_t s) { return n > s ? (n - s - 1) / kStages + 1 : 0u; };
    const uint32_t lane = threadIdx.x & 31;
    if (rank == 0) {
        const uint32_t other = ld_cluster_u32(smem_u32(issued), 1);
        for (uint32_t s = 0; s < kStages; ++s) {
            const uint32_t mine = fills(*issued, s), theirs = fills(other, s), n = max(mine, theirs);
            if (lane == 0 && mine > theirs)
                bar_forgo(full + 8 * s, kStage);
            if (lane == 0 && mine < theirs)
                bar_expect(full + 8 * s, kStage);
            __syncwarp();
            if (n > 0)
                bar_drain(full + 8 * s, (n - 1) & 1);
        }
    }
    const uint32_t c0 = ld_cluster_u32(smem_u32(committed), 0),
                   c1 = ld_cluster_u32(smem_u32(committed + 1), 0);
    for (uint32_t s = 0; s < kStages; ++s)
        if (const uint32_t n = fills(c1, s))
            bar_drain(empty + 8 * s, (n - 1) & 1);
    for (uint32_t b = 0; b < 4; ++b) {
        const uint32_t c = b & 1 ? c1 : c0;
        if (const uint32_t n = (c + 1 - (b >> 1)) / 2)      // sums of even or odd steps
            bar_drain(tfull + 8 * b, (n - 1) & 1);
    }
}

template <class D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    matmul_wide_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_out, MatmulArgs a, int* status,
                       int aligned)
{
    extern __shared__ uint8_t dyn[];
    __shared__ int first_tile[AR_MAX_EXPERTS + 1], first_row[AR_MAX_EXPERTS + 1];
    __shared__ float scale_sh[2][kAhead][2][kHalf];     // two groups of scales
    __shared__ __align__(8) uint64_t bars[2 * kStages + 13];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;
    // for the end of a pair that gave up: whether each block did, copies issued here,
    // products of each half of the columns that the first block committed
    __shared__ uint32_t gave_up_sh[2], issued_sh, committed_sh[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const uint32_t stage0 = (smem_u32(dyn) + 1023u) & ~1023u, out0 = stage0 + kStages * kStage;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages,
                   tempty = tfull + 32, sfull = tempty + 32, sempty = sfull + 16, done = sempty + 16;
    const Bail bail{smem_u32(&dead), status};

    if (tid == 0) {
        dead = 0;
        gave_up_sh[0] = gave_up_sh[1] = 0;
        for (int s = 0; s < kStages; ++s) {
            bar_init(full + 8 * s, 1);      // used in the first block: both blocks' copies
            bar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 4; ++b) {
            bar_init(tfull + 8 * b, 1);
            bar_init(tempty + 8 * b, 8);    // used in the first block: the warps of both
        }
        for (int g = 0; g < 2; ++g) {
            bar_init(sfull + 8 * g, 2);
            bar_init(sempty + 8 * g, 8);
        }
        bar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        if (aligned)
            tma_prefetch_map(&map_out);
    }
    if (warp == 9)
        tmem_alloc_pair(smem_u32(&tmem_slot), kCols);
    pdl_trigger();
    pdl_wait();
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
    __syncwarp();
    tc_fence_before();
    cluster_barrier();          // barriers and tensor memory of both blocks
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int ntn = (a.cols + kN - 1) / kN;
    const int tiles = first_tile[a.experts] * ntn;
    const int nkb = (a.depth + kK - 1) / kK;
    const int t0 = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

    if (warp >= 8) {
        regs_fewer<kRegsIssue>();
        if (warp == 8) {
            uint32_t s = 0, ph = 0, issued = 0;
            bool ok = true;
            const uint32_t full0 = map_rank(full, 0);
            for (int t = t0; t < tiles && ok; t += pairs) {
                const Tile x = tile_at(t, first_tile, first_row, a.experts, ntn);
                const int arow = x.row + kHalf * (int)rank;
                // this block's columns of each half
                const int brow = x.e * a.cols + x.n + kHalf / 2 * (int)rank;
                for (int kb = 0; kb < nkb; ++kb) {
                    ok = __all_sync(0xffffffffu, bar_wait(empty + 8 * s, ph ^ 1, bail, 1));
                    if (!ok)
                        break;
                    if (elect_one()) {
                        const uint32_t at = stage0 + s * kStage;
                        if (rank == 0)
                            bar_expect(full + 8 * s, 2 * kStage);
                        tma_load_pair(at, &map_a, full0 + 8 * s, kb * kK, arow);
                        tma_load_pair(at + kBytes, &map_b, full0 + 8 * s, kb * kK, brow);
                        tma_load_pair(at + kBytes + kBytes / 2, &map_b, full0 + 8 * s, kb * kK,
                                      brow + kHalf);
                    }
                    __syncwarp();
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // until every stage is free again: no copy and no arrival is on its way
            // when the block ends
            for (uint32_t i = 0; i < kStages && i < issued && ok; ++i) {
                const uint32_t back = issued < kStages ? i : (s + i) % kStages;
                const uint32_t par = issued < kStages ? 0u : ((s + i) >= kStages ? ph : ph ^ 1);
                ok = __all_sync(0xffffffffu, bar_wait(empty + 8 * back, par, bail, 1));
            }
            if (lane == 0)
                issued_sh = issued;
        } else if (warp == 9) {
            if (rank == 0 && elect_one()) {
                constexpr uint32_t idesc = fp8_idesc(kM, kN / 2);
                const uint64_t desc0 = smem_desc(stage0);
                const uint32_t hi = (uint32_t)(desc0 >> 32);
                const uint32_t steps = t0 < tiles ? ((tiles - 1 - t0) / pairs + 1) * nkb : 0;
                uint32_t s = 0, ph = 0;
                bool ok = true;
                committed_sh[0] = committed_sh[1] = steps;
                for (uint32_t it = 0; it < steps; ++it) {
                    if (!(ok = bar_wait(full + 8 * s, ph, bail, 3))) {
                        committed_sh[0] = committed_sh[1] = it;
                        break;
                    }
                    const uint32_t at = (uint32_t)desc0 + s * (kStage >> 4);
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        const uint32_t b = 2 * (it & 1) + h;
                        if (!(ok = bar_wait(tempty + 8 * b, (it >> 1 & 1) ^ 1, bail, 2))) {
                            committed_sh[0] = it + h;
                            committed_sh[1] = it;
                            break;
                        }
                        tc_fence_after();
                        mma4_fp8_pair(tmem + b * (kN / 2), at, at + (kBytes >> 4) + h * (kBytes >> 5),
                                      hi, idesc);
                        if (h == 1)
                            mma_commit_pair(empty + 8 * s);
                        mma_commit_pair(tfull + 8 * b);
                    }
                    if (!ok)
                        break;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            __syncwarp();
        } else if (warp >= 10) {
            // two rows per thread, a group of blocks of the depth in flight
            uint32_t grp = 0;
            bool ok = true;
            const int ncb = (a.cols + AR_QUANT_BLOCK - 1) / AR_QUANT_BLOCK;
            for (int t = t0; t < tiles && ok; t += pairs) {
                const Tile x = tile_at(t, first_tile, first_row, a.experts, ntn);
                const int r = 64 * (warp - 10) + lane;
                const int row = x.row + kHalf * (int)rank + r;
                const float* sa0 = a.sa + (uint64_t)(row < x.end ? row : x.row) * nkb;
                const float* sa1 = a.sa + (uint64_t)(row + 32 < x.end ? row + 32 : x.row) * nkb;
                const float* sb0 = a.sb + ((uint64_t)x.e * ncb + x.n / AR_QUANT_BLOCK) * nkb;
                const float* sb1 = x.n + kHalf < a.cols ? sb0 + nkb : sb0;
                for (int kb = 0; kb < nkb && ok; kb += kAhead, ++grp) {
                    float a0[kAhead], a1[kAhead], b0[kAhead], b1[kAhead];
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        const int k = min(kb + j, nkb - 1);
                        a0[j] = sa0[k];
                        a1[j] = sa1[k];
                        b0[j] = sb0[k];
                        b1[j] = sb1[k];
                    }
                    const uint32_t g = grp & 1;
                    ok = __all_sync(0xffffffffu, bar_wait(sempty + 8 * g, (grp >> 1 & 1) ^ 1, bail, 5));
                    if (!ok)
                        break;
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        scale_sh[g][j][0][r] = a0[j] * b0[j];
                        scale_sh[g][j][1][r] = a0[j] * b1[j];
                        scale_sh[g][j][0][r + 32] = a1[j] * b0[j];
                        scale_sh[g][j][1][r + 32] = a1[j] * b1[j];
                    }
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(sfull + 8 * g);
                }
            }
        }
    } else {
        regs_more<kRegsAdd>();
        const int half = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t buf0 = out0 + (uint32_t)warp * kOutBufs * kOutBuf;
        const uint32_t tempty0 = map_rank(tempty, 0);
        // A wait that gives up is not looked at here: the sums are then undefined
        // as the status says, every later wait returns at once, and what is
        // stored stays within the output.
        uint32_t it = 0, grp = 0;
        for (int t = t0; t < tiles; t += pairs) {
            const Tile x = tile_at(t, first_tile, first_row, a.experts, ntn);
            const int row0 = x.row + kHalf * (int)rank + 32 * (warp & 3), row = row0 + lane;
            const int n0 = x.n + 128 * half;
            const bool live = row < x.end && n0 < a.cols;
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i)
                acc[i] = 0ull;
            for (int kb0 = 0; kb0 < nkb; kb0 += kAhead, ++grp) {
                const uint32_t g = grp & 1;
                bar_wait(sfull + 8 * g, grp >> 1 & 1, bail, 6);
                const float* scales = &scale_sh[g][0][half][32 * (warp & 3) + lane];
                float sc = scales[0];
                const int n = min(kAhead, nkb - kb0);
                for (int j = 0; j < n; ++j, ++it) {
                    const uint64_t s2 = pack_pair(__float_as_uint(sc), __float_as_uint(sc));
                    scales += 2 * kHalf;
                    if (j + 1 < n)
                        sc = *scales;
                    const uint32_t b = 2 * (it & 1) + half;
                    bar_wait(tfull + 8 * b, it >> 1 & 1, bail, 4);
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t from = lanes + b * (kN / 2);
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
                                bar_arrive_remote(tempty0 + 8 * b);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            fma_pair(acc[8 * c + i], pack_pair(d[c & 1][2 * i], d[c & 1][2 * i + 1]), s2);
                    }
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(sempty + 8 * g);
            }
            if (n0 >= a.cols || row0 >= x.end)
                continue;
            constexpr int kWords = 16 * D::bytes / 4;
            if (aligned && row0 + 32 <= x.end) {
                // 64 bytes of each of 32 rows at a time through shared memory:
                // stores from registers touch 32 lines each, and the tensor
                // cores waited for them (23 of 118 us at 8192 x 7168 x 2048)
                constexpr int kPer = kOutRow / (16 * D::bytes);     // groups of 16 columns
#pragma unroll
                for (int c = 0; c < 8 / kPer; ++c) {
                    const uint32_t buf = buf0 + (c & 1) * kOutBuf;
                    const int col = n0 + c * (kOutRow / D::bytes);
                    if (col >= a.cols)
                        break;
                    // the first of a tile waits for all: the tile before may have
                    // ended after an odd number, in the same buffer
                    if (lane == 0) {
                        if (c == 0)
                            tma_store_wait_read<0>();
                        else
                            tma_store_wait_read<kOutBufs - 1>();
                    }
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < kPer; ++g) {
                        uint64_t v[8];
                        uint32_t w[kWords];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = acc[8 * (kPer * c + g) + i];
                        round16<D>(v, w);
#pragma unroll
                        for (int i = 0; i < kWords; i += 4) {
                            const uint32_t piece = g * (kWords / 4) + i / 4;
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                             buf + lane * kOutRow + ((piece ^ (lane >> 1 & 3)) << 4)),
                                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3])
                                         : "memory");
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        tma_store_2d(&map_out, buf, col, row0);
                }
            } else if (live) {
                uint8_t* p = static_cast<uint8_t*>(a.out) + ((uint64_t)row * a.cols + n0) * D::bytes;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint64_t v[8];
                    uint32_t w[kWords];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = acc[8 * c + i];
                    round16<D>(v, w);
                    store16<D>(p + 16 * c * D::bytes, w, a.cols - n0 - 16 * c, aligned);
                }
            }
        }
        if (lane == 0)
            tma_store_wait_read<0>();
        __syncwarp();
    }
    __syncthreads();            // every wait that gives up has set the flag
    if (tid == 0 && dead) {
        gave_up_sh[rank] = 1;
        st_cluster_u32(smem_u32(&gave_up_sh[rank]), rank ^ 1, 1);
    }
    __syncwarp();
    tc_fence_before();
    cluster_barrier();
    tc_fence_after();
    // Without a wait that gave up every product has been added and every stage is
    // free again: nothing is on its way.  With one, both blocks know it here, and
    // stay until the last has arrived.
    if (gave_up_sh[0] | gave_up_sh[1]) {
        if (warp == 8)
            end_pair(rank, full, empty, tfull, &issued_sh, committed_sh);
        else if (warp == 9 && rank == 0) {
            if (elect_one())
                mma_commit_pair_here(done);
            __syncwarp();
            bar_drain(done, 0);
        }
        __syncwarp();
        cluster_barrier();
    }
    if (warp == 9)
        tmem_free_pair(tmem, kCols);
}

template <class D>
cudaError_t launch_t(const MatmulArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    CUtensorMap map_a, map_b, map_out = {};
    // stores of whole boxes need rows of 16-byte multiples
    const int aligned = (uint64_t)a.cols * D::bytes % 16 == 0;
    if (!byte_tensor_map(&map_a, a.a, (uint64_t)a.rows, (uint64_t)a.depth, kHalf) ||
        !byte_tensor_map(&map_b, a.b, (uint64_t)a.experts * a.cols, (uint64_t)a.depth,
                         kHalf / 2) ||
        (aligned && !out_tensor_map(&map_out, a.out, (uint64_t)a.rows, (uint64_t)a.cols, D::id, 32,
                                    kOutRow / D::bytes)))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [] {
        // fewer registers at launch than the shares add up to would wait for ever
        cudaFuncAttributes attr;
        const cudaError_t ea = cudaFuncGetAttributes(&attr, matmul_wide_kernel<D>);
        if (ea != cudaSuccess)
            return ea;
        if (attr.numRegs < kRegsLaunch)
            return cudaErrorLaunchOutOfResources;
        return cudaFuncSetAttribute(matmul_wide_kernel<D>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess)
        return e;
    // at most this many tiles: every expert may end in a part of one
    const int64_t most = ((int64_t)a.rows / kM + (a.experts < a.rows ? a.experts : a.rows)) *
                         ((a.cols + kN - 1) / kN);
    if (most > 0x7fffffffll - d.sms)
        return cudaErrorInvalidValue;
    const int pairs = most < d.sms / 2 ? (int)most : d.sms / 2;
    return launch_after(matmul_wide_kernel<D>, 2 * pairs, kThreads, kSmem, s, map_a, map_b, map_out, a,
                        d.status, aligned);
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

// Attention of prompts (any number of new tokens per sequence) over the paged cache.
//
// Scores S = Q K^T and sums O += P V on the tensor cores, both in tensor memory.  The rows
// of a tile are the query heads that share a head of the cache, of consecutive tokens
// (128 / G tokens x G heads, so that a tile's rows see nearly the same keys); a block has
// two tiles, which read the same keys and values from shared memory, 128 keys a step: two
// groups of 64 of those that the rows see (first tokens and window need no step each).
// While the tensor cores work for one tile the four warps of the other turn its
// scores into weights: a thread has a row, so its maximum and sum need no exchange,
// and writes the weights back where the scores were, as the first operand of the
// second product.  The sums are rescaled only where a row's maximum grew far (growth()).
// An item's output is written while the first products of the next one run.
//
//   tensor memory: scores of tile 0, of tile 1, sums of tile 0, of tile 1, 128 columns each
//   warps 0-3, 4-7: softmax and output of tile 0, 1;  warp 8: copies;  warp 9: products;
//   warp 10: clears values that no row sees (what lies there need not be finite);
//   warps 12-15, with a cache of E4M3: turn its codes, which the copies leave beside, into 16-bit
//   keys and values (and clear what no row sees: warp 10 rests);
//   warp 11: finds the items ahead of the others (each for itself took 1.5 us an item)
//
// Items (a pair of tiles and a head) are worked off by one block per SM: where there
// are many, whole ones, dealt out in the order of the sequences (in each the last tokens, which see
// most, first); where there are few, the steps of all items and what the ends of items take (share_of)
// are one list and a block takes an equal share of it.  Items that several blocks
// share are added up by join_kernel from sums, maxima and totals in the workspace.
//
// Long prompts are bound by the tensor cores and the clock that their power leaves: 8192 tokens,
// 32 / 8 heads of 128, bf16: 330 us, 1.66 PFLOP/s of the products that count (0.88 of a library
// product's burst), 1.5 us a step.  With a window of 1024 (3 x 3000-5000 tokens, 64 / 8 heads: 273
// us, 1.17 PFLOP/s) a seventh of the products is of keys that their row does not see, and an item of
// nine steps costs 3 us beside them: masks on its first and last steps, its output.  Chunks of some
// hundred tokens (13 x 40-400 on 600-3000, 14 / 2 heads of 64: 34.5 us) are 14 steps a block, and as
// long again for the start, the ends of the items and the join.
// Over a cache of E4M3 the four warps that widen its codes are the bound: 417 us.
// 64 keys a step with two places for the scores took 450 us instead of 349 (twice the waits for as
// many products), weights ahead of the maximum 27 us more (another pass over the registers).
// Heads of 64 elements: 8192 tokens 282 us, 0.97 PFLOP/s: the products halve, the softmax does not.
// Heads of 72 to 112 elements take the time of 128 (80: 320 us, 96: 331): zeros to 128 in both products.
#include "ar_internal.h"
#include "attention_internal.h"
#include "matmul_internal.h"
#include "tensor_core.cuh"

namespace arf {
namespace {

constexpr int kRows = 128, kKeys = 128, kGroup = 64;   // of a tile, of a step, of a group
// Registers of a thread at launch, of warps 8 on, of warps 0-7.
template <bool F8>
struct Regs {
    static constexpr int threads = F8 ? 512 : 384;
    static constexpr int launch = F8 ? 128 : 168, few = F8 ? 56 : 88, many = F8 ? 200 : 208;
    static_assert((threads / 32 - 8) * few + 8 * many <= threads / 32 * launch, "register shares");
};
constexpr float kLn2 = 0.693147181f;
// How far (in powers of two) a row's maximum may grow before its sums are rescaled: weights are
// then up to 2^growth, as exact as below 1.  A rescaling takes 0.4 us, and with 2^8 some row of
// 32 wanted one in two of three steps of a windowed prompt that begins with a few first tokens.
// The weights are 2^up times e^{s_j - top}.  bf16 ones from 2^-16 to 2^16: the sums of n keys stay
// finite for values below 2^112 / n, and above the denormals for values above 2^-110.
// fp16 weights end at 2^16, have fewer than 11 bits below 2^-14 and nothing below 2^-25: with 2^5 to
// 2^15 for the largest, 2^-30 per key of the sum can be lost (with growth 14 and
// up 0 it was 2^-25, 2^-8 of the sum of 131072 such keys, at 3 x 3000-5000 tokens with a window
// of 1024 and 64 / 8 heads 294 us instead of 303; with 5 and 10 311, and 8192 tokens, 32 / 8
// heads, 369 instead of 337).
template <class D>
__device__ __forceinline__ constexpr float growth() { return D::id == AR_DT_BF16 ? 32.0f : 10.0f; }
template <class D>
__device__ __forceinline__ constexpr float up() { return D::id == AR_DT_BF16 ? -16.0f : 5.0f; }
enum { kWaitStage = 1, kWaitQueryFree, kWaitQuery, kWaitKeys, kWaitWeights, kWaitScores, kWaitSums,
       kWaitCleared, kWaitItem, kWaitPlace };

template <int DP, bool F8 = false>
struct Shape {
    static constexpr int half = kRows * 128;        // bytes of 128 rows of 64 elements
    static constexpr int tile = half * (DP / 64);
    static constexpr int stages = F8 ? (DP == 64 ? 6 : 3) : DP == 64 ? 8 : 4;
    static constexpr int raws = F8 ? (DP == 64 ? 4 : 3) : 0;   // places for codes
    static constexpr int raw = kKeys * DP;
    static constexpr int smem = (2 + stages) * tile + raws * raw + (AR_MAX_SEQUENCES + 1) * 4 + 1024;
    static constexpr int part = 2 * kRows * (DP + 2) * 4;
};
// More than half of an SM's shared memory for every shape: no second block of this kernel
// and no block of the products, which would wait for tensor memory, beside one.
constexpr int kLeastSmem = 200 * 1024;

struct Plan {
    int tok;                    // tokens of a tile
    int whole;                  // 1: items are not split
    int wide;                   // 1: rows of the output are 32-byte aligned
    int4* desc;                 // [blocks]: parts, first row, tokens, head
    uint8_t* parts;             // [blocks][2]
};

// A pair of tiles: tokens from row0 on, `tokens` of them; the first has index i0.
struct Pair {
    int seq, row0, tokens, i0;
    int end, low, sinks;        // keys that any row sees: below end, from low on or below sinks
    int first, gap, groups;     // of 64 keys: the first ones, then those from group first + gap on
    int n;                      // steps of two groups
};

// the first key of group g; behind the last group: one that no row sees
__device__ __forceinline__ int key_of(const Pair& p, int g)
{
    return g < p.groups ? (g < p.first ? g : g + p.gap) * kGroup : p.end;
}
// tokens of a sequence in the call
__device__ __forceinline__ int rows_of(const AttentionArgs& a, int s, int* row0)
{
    const int r0 = a.starts[s], r1 = a.starts[s + 1];
    *row0 = r0;
    return r0 >= 0 && r1 <= a.T && r1 > r0 ? r1 - r0 : 0;
}

// pair f of all: sequences in order, in each the last tokens first
__device__ __forceinline__ Pair pair_at(const AttentionArgs& a, int tok, const int* first_pair, int f)
{
    int lo = 0, hi = a.c.S;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_pair[mid] <= f)
            lo = mid;
        else
            hi = mid;
    }
    Pair p;
    p.seq = lo;
    const int n = rows_of(a, lo, &p.row0);
    const int length = clamp_length(a.c, a.c.lengths[lo]);
    const int t0 = (first_pair[lo + 1] - 1 - f) * 2 * tok;
    p.row0 += t0;
    p.tokens = min(2 * tok, n - t0);
    p.i0 = length - n + t0;
    p.end = max(p.i0 + p.tokens, 0);
    p.low = a.window ? (int)max((long long)p.i0 - a.window + 1, 0ll) : 0;
    p.sinks = a.window ? min(a.sinks, p.end) : 0;
    p.first = (p.sinks + kGroup - 1) / kGroup;
    p.gap = max(0, min(p.low, p.end) / kGroup - p.first);
    p.groups = (p.end + kGroup - 1) / kGroup - p.gap;
    p.n = (p.groups + 1) / 2;
    return p;
}

// What a block does next: steps x0 .. x1 - 1 of a pair for a head (none: nothing left);
// where the item begins here and ends in another block, that block.  Steps clear0 .. clear1 - 1
// hold no key that no row sees.
struct alignas(16) Item {
    Pair p;
    int head, x0, x1, end_block, clear0, clear1;

    __device__ __forceinline__ bool has_unseen(int x) const { return x < clear0 || x >= clear1; }
};
constexpr uint32_t kItems = 4;                      // found ahead

// The items of a block, one after the other.
struct Walk {
    int item, items, x, step;   // whole items: `step` counts them
    int left;                   // of a share: units left (share_of an item's steps)
    int end, total;             // of a share: where it ends in the list, and the list
    int blocks;

    __device__ __forceinline__ bool next(const AttentionArgs& a, const Plan& plan, const int* first_pair,
                                         Item* to)
    {
        for (;;) {
            if (plan.whole) {
                // back and forth over the blocks, so that the first does not get the
                // longest of a sequence in every round
                const long long base = (long long)step * gridDim.x;
                const int at = step & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
                if (base >= items)
                    return false;
                ++step;
                if (base + at >= items)
                    continue;
                item = (int)(base + at);
            } else {
                if (left <= 0)
                    return false;
            }
            const int f = item / a.c.heads;
            to->head = item - f * a.c.heads;
            to->p = pair_at(a, plan.tok, first_pair, f);
            to->x0 = x;
            to->x1 = plan.whole ? to->p.n : min(to->p.n, x + left);
            to->end_block = 0;
            if (!plan.whole) {
                left -= share_of(to->p.n) - x;
                ++item;
                x = 0;
                if (to->x1 < to->p.n)       // the block that has the item's last step
                    to->end_block =
                        (int)(((long long)(end + (to->p.n - to->x1)) * blocks - 1) / total);
            }
            to->clear0 = ((to->p.low + kGroup - 1) / kGroup - to->p.gap + 1) / 2;
            to->clear1 = (to->p.end / kGroup - to->p.gap) / 2;
            if (to->x1 > to->x0)
                return true;
        }
    }
};

// bar_wait in fewer instructions: there are two dozen of them, and with what records the error in
// each the kernel's code did not stay in the instruction caches.  The block's flag holds which
// wait gave up; the end of the kernel records it.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, uint32_t dead, int where)
{
    if (bar_try(bar, parity))
        return true;
    uint32_t t0, t, gave_up;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
    for (uint32_t n = 1; !bar_try(bar, parity); ++n) {
        if (n % ARF_WAIT_TRIES)
            continue;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gave_up) : "r"(dead) : "memory");
        if (gave_up)
            return false;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        if (t - t0 > (uint32_t)ARF_WAIT_NS) {
            asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(dead), "r"(where) : "memory");
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// what a value's code is multiplied with
template <bool F8>
__device__ __forceinline__ float value_scale(const AttentionArgs& a)
{
    return F8 && a.c.scale ? a.c.scale[1] : 1.0f;
}
// the lowest n of 32 bits
__device__ __forceinline__ uint32_t below(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
}

// 16 E4M3 codes as 16-bit elements (exact; a NaN stays one)
template <class D>
__device__ __forceinline__ void widen(const uint4& codes, uint4& lo, uint4& hi)
{
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint16_t two = (uint16_t)(c[i / 2] >> (16 * (i & 1)));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        if constexpr (D::id == AR_DT_BF16) {
            const float2 f = unpack2<Fp16>(h);
            h = pack2<Bf16>(f.x, f.y);
        }
        w[i] = h;
    }
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void put16(uint32_t to, const uint4& v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

template <class D, int DP, bool F8>
__global__ void __launch_bounds__(Regs<F8>::threads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, AttentionArgs a, Plan plan,
                            int* status)
{
    using F = Shape<DP, F8>;
    constexpr uint32_t kStages = F::stages, kRaws = F8 ? F::raws : 1;
    constexpr int kThreads = Regs<F8>::threads;
    constexpr int kTakers = F8 ? 14 : 11;           // warps that take items
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[4 * F::stages + 2 * 7 + 1 + 2 * kItems + 2 * kRaws];
    __shared__ Item item_sh[kItems];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead, begin_sh[2];
    __shared__ int scan_sh[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t q_at = (smem_u32(dyn) + 1023u) & ~1023u, ring = q_at + 2 * F::tile;
    int* first_pair = reinterpret_cast<int*>(dyn + (q_at - smem_u32(dyn)) + (2 + F::stages) * F::tile +
                                             F::raws * F::raw);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, cleared = empty + 8 * kStages,
                   wanted = cleared + 8 * kStages, qfull = wanted + 8 * kStages,
                   qempty = qfull + 16, sfull = qempty + 16, pfull = sfull + 16,
                   ofull = pfull + 32, ofree = ofull + 16, done = ofree + 16,
                   ifull = done + 8, iempty = ifull + 8 * kItems, rfull = iempty + 8 * kItems,
                   rempty = rfull + 8 * kRaws, raw_at = ring + kStages * F::tile;
    const uint32_t bail = smem_u32(&dead);

    if (tid == 0) {
        dead = 0;
        for (uint32_t s = 0; s < kStages; ++s) {
            bar_init(full + 8 * s, F8 ? 4 : 1);
            bar_init(empty + 8 * s, 1);
            bar_init(cleared + 8 * s, 1);
            bar_init(wanted + 8 * s, 1);
        }
        for (int t = 0; t < 2; ++t) {
            bar_init(qfull + 8 * t, 1);
            bar_init(qempty + 8 * t, 1);
            bar_init(sfull + 8 * t, 1);
            bar_init(pfull + 16 * t, 4);        // weights of the first 64 keys, of the others
            bar_init(pfull + 16 * t + 8, 4);
            bar_init(ofull + 8 * t, 1);
            bar_init(ofree + 8 * t, 4);
        }
        bar_init(done, 1);
        for (uint32_t i = 0; F8 && i < kRaws; ++i) {
            bar_init(rfull + 8 * i, 1);
            bar_init(rempty + 8 * i, 4);
        }
        for (uint32_t i = 0; i < kItems; ++i) {
            bar_init(ifull + 8 * i, 1);
            bar_init(iempty + 8 * i, kTakers);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
    }
    if (warp == 9)
        tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before this block has its tensor memory: the next kernel may want some
    pdl_trigger();
    pdl_wait();
    const uint32_t tmem = tmem_slot;

    // pairs before each sequence; whether any has rows without a place.  Starts that decrease
    // could give a row to several sequences, and more pairs than the host reckoned with.
    unsigned before = 0;
    bool short_one = false, falls = false;
#pragma unroll 1
    for (int s0 = 0; s0 < a.c.S; s0 += kThreads) {
        unsigned n = 0;
        if (s0 + tid < a.c.S) {
            int row0;
            n = rows_of(a, s0 + tid, &row0);
            short_one |= clamp_length(a.c, a.c.lengths[s0 + tid]) < (int)n;
            falls |= a.starts[s0 + tid + 1] < row0;
            n = (n + 2 * plan.tok - 1) / (2 * plan.tok);
        }
        unsigned upto = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, upto, m);
            upto += lane >= m ? v : 0;
        }
        if (lane == 31)
            scan_sh[warp] = upto;
        __syncthreads();
        unsigned all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            upto += w < warp ? scan_sh[w] : 0;
            all += scan_sh[w];
        }
        if (s0 + tid < a.c.S)
            first_pair[s0 + tid] = before + upto - n;
        before += all;
        falls = __syncthreads_or(falls);
    }
    const int pairs = falls ? 0 : (int)before;
    if (tid == 0)
        first_pair[a.c.S] = pairs;
    short_one = __syncthreads_or(short_one);

    Walk walk{0, pairs * a.c.heads, 0, 0, 0, 0, 1, (int)gridDim.x};
    if (!plan.whole) {
        // this block's share of the list of units, and where it begins
        const int per = (pairs + kThreads - 1) / kThreads;
        const int f0 = min(tid * per, pairs), f1 = min(f0 + per, pairs);
        int mine = 0, n0 = 0;
#pragma unroll 1
        for (int f = f0; f < f1; ++f) {
            n0 = share_of(pair_at(a, plan.tok, first_pair, f).n);
            mine += n0 * a.c.heads;
        }
        int upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, m);
            upto += lane >= m ? v : 0;
        }
        if (lane == 31)
            scan_sh[warp] = upto;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            upto += w < warp ? scan_sh[w] : 0;
            total += scan_sh[w];
        }
        // no more blocks than units: an item's blocks are then consecutive ones
        const int blocks = min((int)gridDim.x, max(total, 1));
        int u0 = 0;
        walk.total = total;
        walk.blocks = blocks;
        if ((int)blockIdx.x < blocks) {
            // total * block / blocks within 32 bits
            const int each = total / blocks, rest = total - each * blocks;
            u0 = each * blockIdx.x + rest * blockIdx.x / blocks;
            walk.end = each * (blockIdx.x + 1) + rest * (blockIdx.x + 1) / blocks;
            walk.left = walk.end - u0;
        }
        int at = upto - mine;
        if (walk.left && u0 >= at && u0 < upto) {
#pragma unroll 1
            for (int f = f0; f < f1; ++f) {
                const int n = per == 1 ? n0 : share_of(pair_at(a, plan.tok, first_pair, f).n);
                const int end = at + n * a.c.heads;
                if (u0 < end) {
                    const int in = u0 - at;
                    begin_sh[0] = f * a.c.heads + in / n;
                    begin_sh[1] = in % n;
                    break;
                }
                at = end;
            }
        }
        if (tid == 0)
            plan.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        __syncthreads();
        walk.item = begin_sh[0];
        walk.x = begin_sh[1];
    }
    // rows that see nothing, where that holds for a whole pair
#pragma unroll 1
    for (int f = short_one ? (int)blockIdx.x : pairs; f < pairs; f += (int)gridDim.x) {
        const Pair p = pair_at(a, plan.tok, first_pair, f);
        if (p.n > 0)
            continue;
#pragma unroll 1
        for (int i = tid; i < p.tokens * a.Hq; i += kThreads) {
            const int row = p.row0 + i / a.Hq, h = i % a.Hq;
            uint8_t* to = a.out.p + row * a.out.row + h * a.out.head;
#pragma unroll 1
            for (int c = 0; c < a.c.D / 8; ++c)
                *reinterpret_cast<uint4*>(to + 16 * c) = make_uint4(0, 0, 0, 0);
            if (a.lse)
                a.lse[(int64_t)row * a.Hq + h] = -INFINITY;
        }
    }

    // fills of the ring and of the queries' places that warp 8 sent for
    uint32_t sent = 0, asked_for[2] = {0, 0};
    // The next item, by every lane of a warp or by one thread; false: none is left, or a wait gave up.
    Item w;
    uint32_t taken = 0;
    bool ok = true;
    const auto take = [&](bool whole_warp) {
        const uint32_t i = taken % kItems;
        ok = wait_for(ifull + 8 * i, taken / kItems & 1, bail, kWaitItem);
        if (whole_warp)
            ok = __all_sync(0xffffffffu, ok);
        if (!ok)
            return false;
        w = item_sh[i];
        if (whole_warp)
            __syncwarp();
        if (!whole_warp || lane == 0)
            bar_arrive(iempty + 8 * i);
        ++taken;
        return w.x1 > w.x0;
    };
    if (warp >= 8) {
        regs_fewer<Regs<F8>::few>();
        if (warp == 8) {
            // copies: per item the first keys, the queries, then values and keys in turn
            uint32_t it = 0, uses[2] = {0, 0};
            const int page_rows = min(1 << a.c.page_shift, kGroup), boxes = kKeys / page_rows;
            const int box = lane % boxes, part = lane / boxes;      // part: which 64 elements
            while (ok && take(true)) {
#pragma unroll 1
                for (int x = w.x0; x < w.x1 && ok; ++x) {
                    // a lane's box lies in one of the step's two groups
                    const int in = box * page_rows;
                    const int key = key_of(w.p, 2 * x + in / kGroup) + in % kGroup;
                    int page = -1;
                    if (key < w.p.end)
                        page = a.c.table[(int64_t)w.p.seq * a.c.max_pages + (key >> a.c.page_shift)];
                    // outside the map: zeros
                    if (page < 0 || page >= a.c.pages)
                        page = a.c.pages;
                    const int row = page == a.c.pages ? 0 : key & ((1 << a.c.page_shift) - 1);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const uint32_t s = F8 ? it % kRaws : it % kStages;
                        ok = F8 ? wait_for(rempty + 8 * s, (it / kRaws & 1) ^ 1, bail, kWaitStage)
                                : wait_for(empty + 8 * s, (it / kStages & 1) ^ 1, bail, kWaitStage);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
                        if (lane == 0)
                            bar_expect((F8 ? rfull : full) + 8 * s, F8 ? F::raw : F::tile);
                        __syncwarp();
                        // at most 16 boxes a half of the tile
                        if constexpr (F8) {
                            if (part == 0)
                                tma_load_4d(raw_at + s * F::raw + in * DP, kv ? &map_v : &map_k,
                                            rfull + 8 * s, 0, row, w.head, page);
                        } else {
                            const uint32_t to = ring + s * F::tile + in * 128;
                            if (part < DP / 64)
                                tma_load_4d(to + part * F::half, kv ? &map_v : &map_k, full + 8 * s,
                                            64 * part, row, w.head, page);
                        }
                        __syncwarp();
                        // the queries behind the first keys: their place is free later
                        if (x == w.x0 && kv == 0) {
                            for (int t = 0; t < 2 && t * plan.tok < w.p.tokens && ok; ++t) {
                                ok = wait_for(qempty + 8 * t, (uses[t] & 1) ^ 1, bail, kWaitQueryFree);
                                ok = __all_sync(0xffffffffu, ok);
                                if (!ok)
                                    break;
                                if (elect_one()) {
                                    bar_expect(qfull + 8 * t, DP / 64 * 128 * plan.tok * a.G);
                                    for (int h = 0; h < DP / 64; ++h)
                                        tma_load_4d(q_at + t * F::tile + h * F::half, &map_q, qfull + 8 * t,
                                                    64 * h, 0, w.head, w.p.row0 + t * plan.tok);
                                }
                                __syncwarp();
                                ++uses[t];
                            }
                            if (!ok) {
                                ++it;           // the keys are on their way
                                break;
                            }
                        }
                        if (!F8 && kv && lane == 0 && w.has_unseen(x))
                            bar_arrive(wanted + 8 * s);
                    }
                }
            }
            // until every stage and the queries' places are free again: no copy and no arrival is
            // on its way when the block ends
#pragma unroll 1
            for (uint32_t i = it < kStages ? 0 : it - kStages; i < it && ok; ++i)
                ok = __all_sync(0xffffffffu, wait_for(empty + 8 * (i % kStages), i / kStages & 1, bail,
                                                      kWaitStage));
            for (int t = 0; t < 2 && ok; ++t)
                if (uses[t])
                    ok = __all_sync(0xffffffffu, wait_for(qempty + 8 * t, (uses[t] - 1) & 1, bail,
                                                          kWaitQueryFree));
            __syncwarp();
            sent = it;
            asked_for[0] = uses[0];
            asked_for[1] = uses[1];
        } else if (warp == 9) {
            if (elect_one()) {
                constexpr bool bf16 = D::id == AR_DT_BF16;
                constexpr uint32_t id_s = half_idesc(kRows, kKeys, bf16, false);
                constexpr uint32_t id_o = half_idesc(kRows, DP, bf16, true);
                // low words of the descriptors of the queries, and of stage 0 as keys and as values
                const uint64_t desc_k = smem_desc(ring), desc_v = smem_desc_mn(ring, F::half);
                const uint32_t q_lo = (uint32_t)smem_desc(q_at), k_lo = (uint32_t)desc_k,
                               v_lo = (uint32_t)desc_v, k_hi = (uint32_t)(desc_k >> 32),
                               v_hi = (uint32_t)(desc_v >> 32);
                // queries taken, weights taken, items begun (bit t, modulo 2: of tile t)
                uint32_t it = 0, uses = 0, weights = 0, begun = 3, clears = 0;
                const auto landed = [&](uint32_t i) {
                    ok = wait_for(full + 8 * (i % kStages), i / kStages & 1, bail, kWaitKeys);
                    return ok;
                };
                // scores of an item's step from the keys of stage i; of its first step the queries
                // are waited for, behind its last they are done with
                const auto scores = [&](uint32_t t, uint32_t i, bool first, bool last) {
                    if (first) {
                        ok = wait_for(qfull + 8 * t, uses >> t & 1, bail, kWaitQuery);
                        if (!ok)
                            return;
                        uses ^= 1u << t;
                        tc_fence_after();
                    }
                    const uint32_t q = q_lo + t * (F::tile >> 4), k = k_lo + i % kStages * (F::tile >> 4);
#pragma unroll
                    for (int h = 0; h < DP / 64; ++h)
                        mma4_half(tmem + t * 128, q + h * (F::half >> 4), k + h * (F::half >> 4), k_hi, id_s,
                                  h > 0);
                    mma_commit(sfull + 8 * t);
                    if (last)
                        mma_commit(qempty + 8 * t);
                };
                bool more = take(false);
                uint32_t tiles = w.p.tokens > plan.tok ? 2 : 1;
                if (more && landed(it)) {
                    for (uint32_t t = 0; t < tiles && ok; ++t)
                        scores(t, it, true, w.x0 + 1 == w.x1);
                    mma_commit(empty + 8 * (it % kStages));
                    ++it;
                }
                while (ok && more) {
#pragma unroll 1
                    for (int x = w.x0, x0 = x, x1 = w.x1; x < x1 && ok; ++x) {
                        // values of this step: stage it; keys of the next, of the next item behind
                        // the last step: it + 1
                        const uint32_t sv = it % kStages, now = tiles;
                        const bool last = x + 1 == x1, unseen = !F8 && w.has_unseen(x);
                        uint32_t then = tiles;
                        bool next_last = x + 2 == x1;
                        if (last) {
                            more = take(false);
                            tiles = then = !more ? 0 : w.p.tokens > plan.tok ? 2 : 1;
                            next_last = w.x0 + 1 == w.x1;
                            if (!ok)
                                break;
                        }
                        if (!landed(it))
                            break;
                        if (unseen) {
                            if (!(ok = wait_for(cleared + 8 * sv, clears >> sv & 1, bail, kWaitCleared)))
                                break;
                            clears ^= 1u << sv;
                        }
                        const uint32_t v = v_lo + sv * (F::tile >> 4);
                        for (uint32_t t = 0; t < 2; ++t) {
                            if (t < now) {
                                // the sums of the item before have been read
                                if (x == x0) {
                                    if (!(ok = wait_for(ofree + 8 * t, begun >> t & 1, bail, kWaitSums)))
                                        break;
                                    begun ^= 1u << t;
                                }
                                const uint32_t o = tmem + 256 + t * 128, p = tmem + t * 128,
                                               bar = pfull + 16 * t, par = weights >> t & 1;
                                weights ^= 1u << t;
                                if (!(ok = wait_for(bar, par, bail, kWaitWeights)))
                                    break;
                                tc_fence_after();
                                mma4_half_ts(o, p, v, v_hi, id_o, x > x0);
                                if (!(ok = wait_for(bar + 8, par, bail, kWaitWeights)))
                                    break;
                                tc_fence_after();
                                mma4_half_ts(o, p + 32, v + 512, v_hi, id_o, true);
                                if (last)
                                    mma_commit(ofull + 8 * t);
                                if (t + 1 == now)
                                    mma_commit(empty + 8 * sv);
                            }
                            if (t < then) {
                                if (t == 0 && !landed(it + 1))
                                    break;
                                scores(t, it + 1, last, next_last);
                                if (!ok)
                                    break;
                                if (t + 1 == then)
                                    mma_commit(empty + 8 * ((it + 1) % kStages));
                            }
                        }
                        it += then ? 2 : 1;
                    }
                }
            }
            __syncwarp();
        } else if (F8 && warp >= 12) {
            // 16 codes a lane at a time, of 32 keys a warp
            constexpr int kLanes = DP / 16, kStep = 32 / kLanes;    // lanes of a key, keys at a time
            // Loads in flight: the chain of a load, the conversions and the stores, one after the
            // other, took 455 us for 8192 tokens, two at a time 438, four 417, eight spill (496).
            constexpr int kAhead = 4;
            static_assert(32 / kStep % kAhead == 0, "loads ahead");
            const int chunk = lane % kLanes;
            uint32_t it = 0;
            while (ok && take(true)) {
                for (int x = w.x0; x < w.x1 && ok; ++x) {
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const uint32_t r = it % kRaws, s = it % kStages;
                        ok = wait_for(rfull + 8 * r, it / kRaws & 1, bail, kWaitKeys) &&
                             wait_for(empty + 8 * s, (it / kStages & 1) ^ 1, bail, kWaitStage);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
                        const int key0 = key_of(w.p, 2 * x + (warp - 12) / 2) + 32 * (warp & 1);
#pragma unroll
                        for (int i0 = 0; i0 < 32 / kStep; i0 += kAhead) {
                            uint4 codes[kAhead];
#pragma unroll
                            for (int i = 0; i < kAhead; ++i) {
                                const int at = 32 * (warp - 12) + kStep * (i0 + i) + lane / kLanes;
                                uint4& c = codes[i];
                                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(c.x), "=r"(c.y), "=r"(c.z), "=r"(c.w)
                                             : "r"(raw_at + r * F::raw + at * DP + 16 * chunk)
                                             : "memory");
                            }
#pragma unroll
                            for (int i = 0; i < kAhead; ++i) {
                                const int in = kStep * (i0 + i) + lane / kLanes, at = 32 * (warp - 12) + in;
                                const int key = key0 + in;
                                uint4 c = codes[i], lo, hi;
                                // values that no row sees need not be finite
                                if (kv && !(key < w.p.end && (key >= w.p.low || key < w.p.sinks)))
                                    c = make_uint4(0, 0, 0, 0);
                                widen<D>(c, lo, hi);
                                const uint32_t to = ring + s * F::tile + chunk / 4 * F::half + at * 128;
                                const int c0 = chunk % 4 * 2;
                                put16(to + ((c0 ^ (at & 7)) << 4), lo);
                                put16(to + (((c0 + 1) ^ (at & 7)) << 4), hi);
                            }
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            bar_arrive(full + 8 * s);
                            bar_arrive(rempty + 8 * r);
                        }
                    }
                }
            }
        } else if (!F8 && warp == 10) {
            // Values of keys that no row of the pair sees.  The copies say which stage it is: by
            // then the stage's fill before this one is over, so that the wait for the fill is not
            // answered by an older one.
            uint32_t it = 0, asked = 0;
            while (ok && take(true)) {
#pragma unroll 1
                for (int x = w.x0; x < w.x1 && ok; ++x, it += 2) {
                    if (!w.has_unseen(x))
                        continue;
                    const uint32_t s = (it + 1) % kStages;
                    ok = wait_for(wanted + 8 * s, asked >> s & 1, bail, kWaitCleared) &&
                         wait_for(full + 8 * s, (it + 1) / kStages & 1, bail, kWaitKeys);
                    asked ^= 1u << s;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
#pragma unroll 1
                    for (int i = lane; i < kKeys * 8; i += 32) {
                        const int key = key_of(w.p, 2 * x + i / (8 * kGroup)) + i / 8 % kGroup;
                        if (key < w.p.end && (key >= w.p.low || key < w.p.sinks))
                            continue;
#pragma unroll
                        for (int h = 0; h < DP / 64; ++h)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             ring + s * F::tile + h * F::half + i * 16),
                                         "r"(0)
                                         : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(cleared + 8 * s);
                }
            }
        } else if (warp == 11 && lane == 0) {
            // the items, and one without tiles behind the last
#pragma unroll 1
            for (uint32_t i = 0; ok; ++i) {
                if (!(ok = wait_for(iempty + 8 * (i % kItems), (i / kItems & 1) ^ 1, bail, kWaitPlace)))
                    break;
                Item next;
                const bool more = walk.next(a, plan, first_pair, &next);
                if (!more)
                    next.x0 = next.x1 = 0;
                item_sh[i % kItems] = next;
                bar_arrive(ifull + 8 * (i % kItems));
                if (!more)
                    break;
            }
        }
        __syncwarp();
    } else {
        regs_more<Regs<F8>::many>();
        // A wait that gives up is not looked at here: what is stored is then undefined, within the
        // output, and every later wait returns at once.
        const int t = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_at = lanes + t * 128, o_at = lanes + 256 + t * 128;
        const int in = r / a.G, g = r - in * a.G;       // token of the tile, head of the group
        const float scale_log2 = a.scale_log2 * (F8 && a.c.scale ? a.c.scale[0] : 1.0f);
        uint32_t seen = 0, items = 0;
        // the item whose sums are still to be read
        bool held = false;
        float held_top = 0.0f, held_sum = 0.0f;
        int held_row = 0, held_head = 0, held_part = -1;        // row -1: of no token
        const auto give = [&]() {
            held = false;
            wait_for(ofull + 8 * t, items & 1, bail, kWaitSums);
            ++items;
            __syncwarp();
            tc_fence_after();
            const bool live = held_row >= 0;
            const float inv = held_sum > 0.0f || held_sum != held_sum ? value_scale<F8>(a) / held_sum : 0.0f;
            // a warp whose rows are of no token has nothing to say
            const bool any = __any_sync(0xffffffffu, live);
#pragma unroll 1
            for (int c0 = 0; any && c0 < DP; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(o_at + c0, o);
                tmem_wait32(o);
                if (held_part >= 0) {
                    float* part = reinterpret_cast<float*>(
                                      plan.parts + (int64_t)(2 * blockIdx.x + held_part) * F::part) +
                                  (c0 + 2) * 2 * kRows + t * kRows + r;
                    if (live) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            part[c * 2 * kRows] = __uint_as_float(o[c]);
                    }
                    continue;
                }
                uint8_t* to = a.out.p + held_row * a.out.row + held_head * a.out.head + 2 * c0;
#pragma unroll
                for (int c = 0; c < 32; c += 16) {
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = pack2<D>(__uint_as_float(o[c + 2 * e]) * inv,
                                        __uint_as_float(o[c + 2 * e + 1]) * inv);
                    // whole sectors where the output allows it
                    const int n = a.c.D - c0 - c;
                    if (plan.wide && n >= 16) {
                        if (live)
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + 2 * c),
                                         "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                                         "r"(v[6]), "r"(v[7])
                                         : "memory");
                    } else {
                        if (live && n > 0)
                            *reinterpret_cast<uint4*>(to + 2 * c) = make_uint4(v[0], v[1], v[2], v[3]);
                        if (live && n > 8)
                            *reinterpret_cast<uint4*>(to + 2 * c + 16) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(ofree + 8 * t);
            if (!live)
                return;
            if (held_part >= 0) {
                float* part = reinterpret_cast<float*>(
                                  plan.parts + (int64_t)(2 * blockIdx.x + held_part) * F::part) +
                              t * kRows + r;
                part[0] = held_top;
                part[2 * kRows] = held_sum;
            } else if (a.lse) {
                a.lse[(int64_t)held_row * a.Hq + held_head] = (held_top + log2f(held_sum)) * kLn2;
            }
        };
        while (take(true)) {
            const int tok0 = t * plan.tok;
            if (tok0 >= w.p.tokens)
                continue;
            const bool live = in < plan.tok && tok0 + in < w.p.tokens;
            const int i = live ? w.p.i0 + tok0 + in : -1;
            const int ia = w.p.i0 + tok0, ib = w.p.i0 + min(tok0 + plan.tok, w.p.tokens) - 1;
            // steps full0 .. full1 - 1: every row sees every key
            const int full0 = a.window ? (max(ib - a.window + kGroup, 0) / kGroup - w.p.gap + 1) / 2 : 0,
                      full1 = (max(ia + 1, 0) / kGroup - w.p.gap) / 2;
            float top = -INFINITY;
            uint64_t sum = 0;
#pragma unroll 1
            for (int x = w.x0; x < w.x1; ++x, ++seen) {
                wait_for(sfull + 8 * t, seen & 1, bail, kWaitScores);
                __syncwarp();
                tc_fence_after();
                uint32_t s[kKeys];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(s_at + 32 * c, s + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_wait32(s + 32 * c);
                if (__builtin_expect(x < full0 || x >= full1, 0)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key0 = key_of(w.p, 2 * x + h);
                        const int hi = i + 1 - key0, lo = a.window ? i - a.window + 1 - key0 : 0,
                                  first = a.sinks - key0;
#pragma unroll
                        for (int c = 0; c < kGroup; c += 32) {
                            const uint32_t bits = below(hi - c) & (~below(lo - c) | below(first - c));
                            if (__all_sync(0xffffffffu, bits == 0xffffffffu))
                                continue;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[kGroup * h + c + e] = bits >> e & 1 ? s[kGroup * h + c + e] : 0xff800000u;
                        }
                    }
                }
                float m[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    m[c] = max3(__uint_as_float(s[3 * c]), __uint_as_float(s[3 * c + 1]),
                                __uint_as_float(s[3 * c + 2]));
#pragma unroll
                for (int c = 12; c < kKeys; c += 2)
                    m[c / 2 & 3] = max3(m[c / 2 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                const float best = fmaxf(max3(m[0], m[1], m[2]), m[3]) * scale_log2;
                if (__builtin_expect(__any_sync(0xffffffffu, best > top + growth<D>()), 0)) {
                    const float now = best > top + growth<D>() ? best : top;
                    const float f = now == top ? 1.0f : exp2_fast(top - now);
                    top = now;
                    sum = mul_pair(sum, pair_of(f, f));
                    if (x > w.x0) {
#pragma unroll 1
                        for (int c = 0; c < DP; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_at + c, o);
                            tmem_wait(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(o_at + c, o);
                        }
                    }
                }
                // The products of the first half of the weights begin while the second half is made.
                const float used = top == -INFINITY ? 0.0f : top;
                const uint64_t scale = pair_of(scale_log2, scale_log2), minus = pair_of(up<D>() - used, up<D>() - used);
                uint64_t part[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int k = 64 * h + 2 * e;
                        const float2 z = unpack_pair(fma3_pair(pack_pair(s[k], s[k + 1]), scale, minus));
                        const float e0 = exp2_fast(z.x), e1 = exp2_fast(z.y);
                        part[e & 3] = add_pair(part[e & 3], pair_of(e0, e1));
                        p[e] = pack2<D>(e0, e1);
                    }
                    tmem_st32(s_at + 32 * h, p);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(pfull + 16 * t + 8 * h);
                }
                sum = add_pair(sum, add_pair(add_pair(part[0], part[1]), add_pair(part[2], part[3])));
                if (__builtin_expect(held, 0))
                    give();
            }
            const float2 two = unpack_pair(sum);
            held = true;
            held_top = top - up<D>();
            held_sum = two.x + two.y;
            held_row = live ? w.p.row0 + tok0 + in : -1;
            held_head = w.head * a.G + g;
            // a piece that begins here is part 1, one that began before part 0
            held_part = w.x0 > 0 ? 0 : w.x1 < w.p.n ? 1 : -1;
            if (held_part == 1 && tid == 0)
                plan.desc[blockIdx.x] = make_int4(w.end_block - (int)blockIdx.x + 1, w.p.row0, w.p.tokens,
                                                  w.head);
        }
        if (held)
            give();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Without a wait that gave up every product has been taken and every copy is consumed.
    // With one, whichever warp's it was, both end here before the block does.
    if (const int where = *static_cast<volatile int*>(&dead)) {
        if (tid == 0 && atomicCAS(status, 0, AR_ERR_TIMEOUT) == 0)
            atomicExch(status + 1, where);
        if (warp == 8) {
            constexpr uint32_t kPlaces = F8 ? kRaws : kStages;
#pragma unroll 1
            for (uint32_t i = sent < kPlaces ? 0 : sent - kPlaces; i < sent; ++i)
                bar_drain((F8 ? rfull : full) + 8 * (i % kPlaces), i / kPlaces & 1);
            for (int t = 0; t < 2; ++t)
                if (asked_for[t])
                    bar_drain(qfull + 8 * t, (asked_for[t] - 1) & 1);
        } else if (warp == 9) {
            if (elect_one())
                mma_commit(done);
            __syncwarp();
            bar_drain(done, 0);
        }
    }
    if (warp == 9)
        tmem_free(tmem, 512);
}

// Items that several blocks share.  Block (b, y): the item that begins in block b, 8 of its
// elements; a thread has a row, and all of its loads of kJoinAhead parts in flight.
constexpr int kJoinAhead = 4, kJoinDims = 8;

template <class D, int DP>
__global__ void __launch_bounds__(2 * kRows) join_kernel(AttentionArgs a, Plan plan)
{
    pdl_trigger();
    pdl_wait();
    const int4 d = plan.desc[blockIdx.x];
    const int r = threadIdx.x, in = r % kRows / a.G, g = r % kRows - in * a.G;
    const int token = r / kRows * plan.tok + in, d0 = blockIdx.y * kJoinDims;
    if (d.x == 0 || in >= plan.tok || token >= d.z || d0 >= a.c.D)
        return;
    float m = -INFINITY, l = 0.0f, acc[kJoinDims];
#pragma unroll
    for (int e = 0; e < kJoinDims; ++e)
        acc[e] = 0.0f;
    for (int p0 = 0; p0 < d.x; p0 += kJoinAhead) {
        float pm[kJoinAhead], pl[kJoinAhead], v[kJoinAhead][kJoinDims];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const int p = p0 + i;
            const int slot = p == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + p);
            const float* s =
                reinterpret_cast<const float*>(plan.parts + (int64_t)slot * Shape<DP>::part) + r;
            pm[i] = p < d.x ? s[0] : -INFINITY;
            pl[i] = p < d.x ? s[2 * kRows] : 0.0f;
#pragma unroll
            for (int e = 0; e < kJoinDims; ++e)
                v[i][e] = p < d.x ? s[(2 + d0 + e) * 2 * kRows] : 0.0f;
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            top = fmaxf(top, pm[i]);
        const float base = top == -INFINITY ? 0.0f : top, f = exp2_fast(m - base);
        l *= f;
#pragma unroll
        for (int e = 0; e < kJoinDims; ++e)
            acc[e] *= f;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const float wt = exp2_fast(pm[i] - base);
            l = fmaf(pl[i], wt, l);
#pragma unroll
            for (int e = 0; e < kJoinDims; ++e)
                acc[e] = fmaf(v[i][e], wt, acc[e]);
        }
        m = top;
    }
    const float inv = l > 0.0f || l != l ? value_scale<true>(a) / l : 0.0f;     // no scale: 1
    const int row = d.y + token, h = d.w * a.G + g;
#pragma unroll
    for (int e = 0; e < kJoinDims; ++e)
        acc[e] *= inv;
    *reinterpret_cast<uint4*>(a.out.p + row * a.out.row + h * a.out.head + 2 * d0) = pack8<D>(acc);
    if (a.lse && blockIdx.y == 0)
        a.lse[(int64_t)row * a.Hq + h] = (m + log2f(l)) * kLn2;
}

// the stride of an extent of one: any multiple of 16
uint64_t stride_of(int64_t stride) { return stride ? (uint64_t)stride : 16u; }

template <class D, int DP, bool F8>
cudaError_t launch_t(const AttentionArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    constexpr int smem = Shape<DP, F8>::smem > kLeastSmem ? Shape<DP, F8>::smem : kLeastSmem;
    static_assert(smem <= 227 * 1024 - 2048, "shared memory");
    Plan plan{};
    plan.tok = kRows / a.G;
    plan.wide = ((uintptr_t)a.out.p | (uint64_t)a.out.row | (uint64_t)a.out.head) % 32 == 0;
    const uint64_t D_ = (uint64_t)a.c.D;
    const uint32_t page = 1u << a.c.page_shift, box = page < (uint32_t)kGroup ? page : kGroup;
    CUtensorMap map_q, map_k, map_v;
    const int type = F8 ? (int)AR_DT_E4M3 : D::id;
    const uint32_t wide = F8 ? DP : 64;
    if (!rows_tensor_map(&map_q, D::id, a.q.p, {D_, (uint64_t)a.G, (uint64_t)a.c.heads, (uint64_t)a.T},
                         {stride_of(a.q.head), stride_of(a.q.head * a.G), stride_of(a.q.row)},
                         {64, (uint32_t)a.G, 1, (uint32_t)plan.tok}) ||
        !rows_tensor_map(&map_k, type, a.c.k, {D_, page, (uint64_t)a.c.heads, (uint64_t)a.c.pages},
                         {stride_of(a.c.k_row), stride_of(a.c.k_head), stride_of(a.c.k_page)},
                         {wide, box, 1, 1}) ||
        !rows_tensor_map(&map_v, type, a.c.v, {D_, page, (uint64_t)a.c.heads, (uint64_t)a.c.pages},
                         {stride_of(a.c.v_row), stride_of(a.c.v_head), stride_of(a.c.v_page)},
                         {wide, box, 1, 1}))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        // fewer registers at launch than the shares add up to would wait for ever
        cudaFuncAttributes attr;
        const cudaError_t ea = cudaFuncGetAttributes(&attr, prompt_attention_kernel<D, DP, F8>);
        if (ea != cudaSuccess)
            return ea;
        if (attr.numRegs < Regs<F8>::launch)
            return cudaErrorLaunchOutOfResources;
        return cudaFuncSetAttribute(prompt_attention_kernel<D, DP, F8>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess)
        return e;
    // at most so many items: every sequence may end in a part of a pair
    const int64_t items = ((int64_t)a.T / (2 * plan.tok) + (a.c.S < a.T ? a.c.S : a.T)) * a.c.heads;
    if (items > 0x7fffffffll - d.sms)
        return cudaErrorInvalidValue;
    int blocks = d.sms;
    const int64_t fit = (int64_t)(a.work_bytes / (16 + 2 * Shape<DP>::part));
    const int64_t keys = (int64_t)a.c.max_pages << a.c.page_shift;
    const int64_t steps = items * ((keys + kKeys - 1) / kKeys + 1);     // at most
    // Whole items or equal shares.  The host knows neither lengths nor how many items there are, only
    // the most there can be.  From four an SM on they are dealt out whole: a prompt of 8192 tokens, 32 /
    // 8 heads, 330 us; but one of 131072 among 127 of 1000, 4 new tokens each, 64 / 8 heads, is one
    // block's work, 1267 us where its bytes take 158.  Below that shares win where lengths are uneven
    // or new tokens few (60 x 4 on 500-32000, 64 / 8 heads, 306 us, whole 367; 512 behind 4000, 32 / 8
    // heads, 43 and 56), whole items for prompts without a cached part (3000 tokens, 32 / 8 heads, 60,
    // in shares 78; 700, twice, 17.5 and 27).
    // A workspace for much fewer blocks than whole items keep busy would slow the call down (512
    // behind 4000, 72 items: 31 blocks 115 us, 63 blocks 64, whole 56; the three quarters
    // leave AR_ATTENTION_WORKSPACE_BYTES' 126 blocks of 152).
    const int64_t busy = items < d.sms ? items : d.sms;
    plan.whole = items >= 4ll * d.sms || fit < 2 || 4 * fit < 3 * busy ||
                 steps + kItemEnd * items >= 1 << 30;
    if (plan.whole) {
        if (items < blocks)
            blocks = (int)items;
    } else {
        // no block for an item's end alone, where there is one for each step
        if (steps < blocks)
            blocks = (int)steps;
        if (fit < blocks)
            blocks = (int)fit;
        plan.desc = reinterpret_cast<int4*>(a.work);
        plan.parts = a.work + 16 * (int64_t)blocks;
    }
    const bool joined = !plan.whole && blocks > 1;
    std::unique_lock<std::mutex> both(launches_with(a.work), std::defer_lock);
    if (joined)
        both.lock();
    e = launch_after(prompt_attention_kernel<D, DP, F8>, blocks, Regs<F8>::threads, smem, s, map_q, map_k,
                     map_v, a, plan, d.status + kStatusWords);
    if (e != cudaSuccess || !joined)
        return e;
    return launch_after(join_kernel<D, DP>, dim3(blocks, DP / kJoinDims), 2 * kRows, 0, s, a, plan);
}

template <class D>
cudaError_t launch_d(bool e4m3, const AttentionArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    if (a.c.D <= 64)
        return e4m3 ? launch_t<D, 64, true>(a, d, s) : launch_t<D, 64, false>(a, d, s);
    return e4m3 ? launch_t<D, 128, true>(a, d, s) : launch_t<D, 128, false>(a, d, s);
}

}  // namespace

cudaError_t launch_prompt_attention(int dtype, bool e4m3, const AttentionArgs& a, cudaStream_t s)
{
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess)
        return e;
    return dtype == AR_DT_BF16 ? launch_d<Bf16>(e4m3, a, d, s) : launch_d<Fp16>(e4m3, a, d, s);
}

}  // namespace arf

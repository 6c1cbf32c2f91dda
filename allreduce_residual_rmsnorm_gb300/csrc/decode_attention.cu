// Attention of one new token per sequence over the paged cache.
//
// Memory bounds it: every key and value is read once for each 16 of the query heads that
// share it.  Those are the 8 columns of m16n8k16 products (two of them for 9 to 16 heads):
// S^T = K Q^T, O^T = V^T P^T, keys and values straight from shared memory as first operands, the
// weights turned by movmatrix from one product's result to the next one's operand.
// With the heads as the 16 rows, half of them empty at 8, the products of an E4M3 cache
// took longer than its bytes (128 x 2048-4096 tokens x 64 / 8 heads 180 us).  At 8 heads per
// key the arithmetic is 8 operations a byte, 54 T a second at the memory's rate: more
// than the fp32 pipes have left beside the conversions, little for these products;
// the instructions on 128 rows of tensor memory would waste seven eighths of them and
// pay a round trip to it for every tile.
//
// A warp has slices of its own: 4 KB of keys and 4 KB of values, a ring of kStages of
// them filled by asynchronous copies, a running maximum and sum, and its own sums.
// (Tensor-map copies, one thread's, were 3% faster for E4M3 and 5 to 6% slower for 16 bits.)
// Four warps take the four slices of a unit in turn and meet at the end of a piece.
//
// All units of all sequences and heads are one list; a block takes an equal share of it
// wherever that begins and ends, so uneven lengths leave no block behind.  A block
// holds whole items, and at most two pieces of items that other blocks share: those go
// to the workspace as sums, maximum and total, and join_kernel, launched behind it,
// adds them in the order of the blocks.
//
// 64 x 800-8000 tokens, 32 / 8 heads, bf16: 173 to 180 us, 6.4 to 6.7 TB/s (0.95 to 0.98 of a
// copy); one sequence of 131072, 64 / 8 heads: 84 us, 6.4 TB/s; E4M3, 128 x 2048-4096, 64 / 8
// heads: 133 to 143 us, 5.7 to 6.1 TB/s, what is left goes to the widening of the codes (issue
// slots 55% used).  4 x 500-1000 tokens, 8 / 1 heads: 7.6 us, two launches and two reads behind
// one another (page number, keys) with a join.  33 windows of 1000, 28 / 4 heads of 80: 16.3 us: a
// block has some ten units, and the one that stands for an item's end has no slice, so that a place
// of the ring is empty whenever an item ends.
// 9 to 16 heads per key: 64 x 800-8000 tokens, 64 / 4 heads, 99 us, 5.8 TB/s; E4M3, 128 / 8 heads, 176,
// 4.6 TB/s (twice the weights and products for the bytes).  More read the keys again for every
// 16: 32 x 8000, 16 / 1 heads 30 us, 32 / 1 49, 64 / 1 86, 128 / 1 161.
#include "ar_internal.h"
#include "attention_internal.h"
#include "matmul_internal.h"
#include "tensor_core.cuh"

namespace arf {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 4096;             // bytes of keys, and of values, of a slice
constexpr int kRows = 16;               // query heads of an item
constexpr float kLn2 = 0.693147181f;

// Blocks on an SM and slices in a warp's ring.  Two of three slices hold more bytes in flight than
// three of two; but the codes of an E4M3 slice of the same bytes are twice the work, and want
// the warps (147 -> 133 us, 5.5 -> 6.1 TB/s; 16 bits 83.4 -> 88.0 the other way, 131072 tokens).
template <bool F8, int NB>
struct Fit {
    static constexpr int blocks = F8 && NB == 1 ? 3 : 2, stages = F8 && NB == 1 ? 2 : 3;
};

struct Split {
    int4* desc;                         // [blocks]: parts, sequence, head, tile
    uint8_t* parts;                     // [blocks][2] of part_bytes
    int whole;                          // 1: items are not split
};
template <int DP>
__host__ __device__ constexpr int part_bytes()
{
    return 2 * kRows * 4 + kRows * DP * 4;      // maxima, totals, sums in the order of fragments
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there)
{
    const int n = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// the 8 x 8 matrix of 16-bit elements that a warp holds, turned over
__device__ __forceinline__ uint32_t turned(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void ldm4_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two E4M3 codes of the low 16 bits as two fp16 values (exact)
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

// What of a sequence's cache the token sees, in slices: the first `sinks` and from `low`
// on; slice x of `n` is x, or x + gap behind the first ones.
struct Seen {
    int length, low, sinks, first, gap, n;
};
template <int SL>
__device__ __forceinline__ Seen seen_of(const AttentionArgs& a, int length)
{
    Seen s;
    s.length = clamp_length(a.c, length);
    s.low = a.window ? max(0, s.length - a.window) : 0;
    s.sinks = min(a.sinks, s.length);
    s.first = (s.sinks + SL - 1) / SL;
    const int end = (s.length + SL - 1) / SL, from = s.low / SL;
    s.gap = max(0, from - s.first);
    s.n = end - s.gap;
    return s;
}

// Units of an item: of four slices, and one more for its end, which takes as long: without it
// blocks with many short items were the last by far (33 windows of 1000 21.6 us, now 17.1).
__device__ __forceinline__ int units_of(const Seen& s)
{
    return s.n ? (s.n + kWarps - 1) / kWarps + 1 : 0;
}

// A place in the list of units: unit `unit` of `units` of tile `tile` of the query heads of head
// `head` of sequence `seq`.  (Without divisions: a warp is one chain of instructions, and each
// would be a tenth of a unit.)
template <int SL>
struct Cursor {
    int seq, head, tile, unit, units;
    const int32_t* table;       // of the sequence
    int after;                  // length of the next sequence, asked for ahead
    Seen seen;

    __device__ __forceinline__ void enter(const AttentionArgs& a, int s, int length)
    {
        seq = s;
        table = a.c.table + (int64_t)s * a.c.max_pages;
        after = s + 1 < a.c.S ? a.c.lengths[s + 1] : 0;
        seen = seen_of<SL>(a, length);
        units = units_of(seen);
    }
    // to the next unit, while there is one
    __device__ __forceinline__ void next(const AttentionArgs& a, int tiles)
    {
        if (++unit < units)
            return;
        unit = 0;
        if (++tile < tiles)
            return;
        tile = 0;
        if (++head < a.c.heads)
            return;
        head = 0;
        do {
            if (seq + 1 == a.c.S)       // the end of the list: not used further
                return;
            enter(a, seq + 1, after);
        } while (units == 0);
    }
};

template <class D, int DP, bool F8>
struct Form {
    static constexpr int bytes = F8 ? 1 : 2;            // of an element of the cache
    static constexpr int pitch = (DP <= 64 ? 64 : 128) * bytes;     // of a slice's row
    static constexpr int SL = kTile / pitch;            // keys of a slice
    static constexpr bool bf16 = !F8 && D::id == AR_DT_BF16;    // products' type
    // The weights are 2^up times e^{s_j - max}.  fp16 keeps 11 bits down to 2^-14 only and nothing
    // below 2^-25: of 131072 keys whose weights are 2^-25 each a share of 2^-8 was lost.  With 2^14
    // for the largest all are kept to 2^-39.
    static constexpr float up = bf16 ? 0.0f : 14.0f;
    // 16-byte chunk `c` of row r: the 8 rows of a matrix load in different banks
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        return r * pitch + ((pitch == 64 ? c ^ (r >> 1 & 3) : c ^ (r & 7)) << 4);
    }
};

// First key of the slice of a warp in a cursor's unit; -1: it has none.
template <int SL>
__device__ __forceinline__ int slice_key(const Cursor<SL>& c, int warp)
{
    const int x = c.unit * kWarps + warp;
    return x < c.seen.n ? (x < c.seen.first ? x : x + c.seen.gap) * SL : -1;
}
// The page of 8 keys of that slice, by lane; -1: none.  Asked for a unit before its copies: with
// the two together the answer's way, 0.7 us, was half of the time of a unit.
template <int SL>
__device__ __forceinline__ int slice_page(const AttentionArgs& a, const Cursor<SL>& c, int warp, int lane)
{
    const int key0 = slice_key(c, warp), mine = key0 + 8 * lane;
    if (key0 < 0 || lane >= SL / 8 || mine >= c.seen.length)
        return -1;
    return c.table[mine >> a.c.page_shift];
}
// Copies of one slice into a stage, by one warp: a lane has a chunk of every kStep-th row.
template <class F>
__device__ __forceinline__ void load_slice(const AttentionArgs& a, int key0, int head, int page, int lane,
                                           uint32_t stage)
{
    if (key0 >= 0) {
        constexpr int kChunks = F::pitch / 16, kStep = 32 / kChunks;
        const int chunk = lane % kChunks, row = lane / kChunks, mask = (1 << a.c.page_shift) - 1;
        if (page >= a.c.pages)
            page = -1;
        const uint8_t* k = a.c.k + head * a.c.k_head + chunk * 16;
        const uint8_t* v = a.c.v + head * a.c.v_head + chunk * 16;
        const bool used = chunk * 16 < a.c.D * F::bytes;
#pragma unroll
        for (int i = 0; i < kTile / 512; ++i) {
            const int r = i * kStep + row, in = (key0 + r) & mask;
            const int p = __shfl_sync(0xffffffffu, page, r >> 3);
            const bool there = p >= 0;
            const int64_t pp = max(p, 0);
            if (used) {
                const uint32_t to = stage + F::at(r, chunk);
                copy16(to, k + (pp * a.c.k_page + in * a.c.k_row), there);
                copy16(to + kTile, v + (pp * a.c.v_page + in * a.c.v_row), there);
            }
        }
    }
    copies_commit();
}

// Register (tile j of 16 elements, n of 8 heads, e) of a thread's sums: which element of
// the head, and which head.
template <bool F8>
__device__ __forceinline__ int dim_of(int j, int e, int g)
{
    return 16 * j + (F8 ? 2 * g + (e >> 1) : g + 8 * (e >> 1));
}
__device__ __forceinline__ int head_of(int n, int e, int t) { return 8 * n + 2 * t + (e & 1); }

// a thread's two elements of tile j of a head
template <class D, bool F8>
__device__ __forceinline__ void store_dims(uint8_t* to, int dims, int j, int g, float f0, float f1)
{
    const uint32_t v = pack2<D>(f0, f1);
    const int d0 = dim_of<F8>(j, 0, g), d1 = dim_of<F8>(j, 2, g);
    if constexpr (F8) {
        if (d0 < dims)          // even: the next one is in, too
            *reinterpret_cast<uint32_t*>(to + 2 * d0) = v;
    } else {
        if (d0 < dims)
            *reinterpret_cast<uint16_t*>(to + 2 * d0) = (uint16_t)v;
        if (d1 < dims)
            *reinterpret_cast<uint16_t*>(to + 2 * d1) = (uint16_t)(v >> 16);
    }
}

template <class D, int DP, bool F8, int NB>
__global__ void __launch_bounds__(kThreads, Fit<F8, NB>::blocks)
    decode_attention_kernel(AttentionArgs a, Split sp, int tiles)
{
    using F = Form<D, DP, F8>;
    constexpr int SL = F::SL, NK = SL / 16, KS = DP / 16, kStages = Fit<F8, NB>::stages;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ float max_sh[kWarps][kRows], sum_sh[kWarps][kRows];
    __shared__ long long scan_sh[kWarps], where_sh[2];
    __shared__ int begin_sh[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int heads = a.c.heads * tiles;        // items of a sequence
    float* sums = reinterpret_cast<float*>(dyn + kWarps * kStages * 2 * kTile);
    const uint32_t ring = smem_u32(dyn) + warp * kStages * 2 * kTile;
    pdl_trigger();
    // chunks behind the head's last element are never copied: zero once, for good
    if (DP > a.c.D)
        for (int i = tid; i < kWarps * kStages * 2 * kTile / 16; i += kThreads)
            reinterpret_cast<uint4*>(dyn)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();

    // this block's share of the list of units, and where it begins
    const int per = (a.c.S + kThreads - 1) / kThreads;
    const int s0 = min(tid * per, a.c.S), s1 = min(s0 + per, a.c.S);
    long long mine = 0;
#pragma unroll 1
    for (int s = s0; s < s1; ++s)
        mine += (long long)units_of(seen_of<SL>(a, a.c.lengths[s])) * heads;
    long long upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, m);
        upto += lane >= m ? v : 0;
    }
    if (lane == 31)
        scan_sh[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        upto += w < warp ? scan_sh[w] : 0;
        total += scan_sh[w];
    }
    // no more blocks than units: an item's blocks are then consecutive ones
    const int block = blockIdx.x, blocks = (int)min((long long)gridDim.x, max(total, 1ll));
    long long u0 = total, u1 = total;
    if (block < blocks) {
        if (total < 1ll << 31) {        // total * block / blocks in 32 bits
            const unsigned each = (unsigned)total / (unsigned)blocks,
                           rest = (unsigned)total - each * (unsigned)blocks;
            u0 = each * block + rest * block / (unsigned)blocks;
            u1 = each * (block + 1) + rest * (block + 1) / (unsigned)blocks;
        } else {
            u0 = total * block / blocks;
            u1 = total * (block + 1) / blocks;
        }
    }
    if (sp.whole) {
        // items whose first unit lies in the share
        if (tid < 2)
            where_sh[tid] = total;
        __syncthreads();
        long long at = upto - mine;
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            const int n = units_of(seen_of<SL>(a, a.c.lengths[s]));
            const long long end = at + (long long)n * heads;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const long long u = i ? u1 : u0;
                // the first item that starts at u or behind it
                if (n && u <= end - n)
                    atomicMin(&where_sh[i], u <= at ? at : at + (u - at + n - 1) / n * n);
            }
            at = end;
        }
        __syncthreads();
        u0 = where_sh[0];
        u1 = where_sh[1];
    }
    {
        long long at = upto - mine;
        if (u0 < u1 && u0 >= at && u0 < upto) {
#pragma unroll 1
            for (int s = s0; s < s1; ++s) {
                const int n = units_of(seen_of<SL>(a, a.c.lengths[s]));
                const long long end = at + (long long)n * heads;
                if (u0 < end) {
                    const UnitPlace p = unit_place(u0 - at, n);
                    begin_sh[0] = s;
                    begin_sh[1] = p.item;
                    begin_sh[2] = p.unit;
                    break;
                }
                at = end;
            }
        }
    }
    // sequences without a key
#pragma unroll 1
    for (int s = block; s < a.c.S; s += (int)gridDim.x) {
        if (seen_of<SL>(a, a.c.lengths[s]).n > 0)
            continue;
#pragma unroll 1
        for (int h = tid; h < a.Hq; h += kThreads) {
            uint8_t* to = a.out.p + s * a.out.row + h * a.out.head;
#pragma unroll 1
            for (int c = 0; c < a.c.D / 8; ++c)
                *reinterpret_cast<uint4*>(to + 16 * c) = make_uint4(0, 0, 0, 0);
            if (a.lse)
                a.lse[(int64_t)s * a.Hq + h] = -INFINITY;
        }
    }
    if (tid == 0 && !sp.whole)
        sp.desc[block] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (u0 >= u1)
        return;

    Cursor<SL> c, ahead;
    c.enter(a, begin_sh[0], a.c.lengths[begin_sh[0]]);
    c.head = begin_sh[1] / tiles;
    c.tile = begin_sh[1] - c.head * tiles;
    c.unit = begin_sh[2];
    ahead = c;
    const long long count = u1 - u0;
    float k_scale = 1.0f, v_scale = 1.0f;
    if (F8 && a.c.scale) {
        k_scale = a.c.scale[0];
        v_scale = a.c.scale[1];
    }
    int page = slice_page(a, ahead, warp, lane);
    const auto send = [&](int to) {
        const int key0 = slice_key(ahead, warp), head = ahead.head, its = page;
        ahead.next(a, tiles);
        page = slice_page(a, ahead, warp, lane);
        load_slice<F>(a, key0, head, its, lane, ring + to * 2 * kTile);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < count)
            send(i);
        else
            copies_commit();
    }

    uint32_t q[KS][NB][2];
    float o[KS][NB][4];
    float top[NB][2], total_w[NB][2], factor[NB][2];
    bool fresh = true, whole_start = c.unit == 0;
    int stage = 0;
#pragma unroll 1
    for (long long u = 0; u < count; ++u) {
        const int rows = min(kRows, a.G - c.tile * kRows);
        const int q_head = c.head * a.G + c.tile * kRows;
        if (fresh) {
            fresh = false;
            const uint8_t* qp = a.q.p + c.seq * a.q.row + q_head * a.q.head;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const uint8_t* qh = qp + (8 * n + g) * a.q.head;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int d = F8 ? 16 * ks + 4 * t + 2 * half : 16 * ks + 8 * half + 2 * t;
                        const bool in = (F8 ? 16 * ks : 16 * ks + 8 * half) < a.c.D;
                        q[ks][n][half] = in && 8 * n + g < rows
                                             ? *reinterpret_cast<const uint32_t*>(qh + 2 * d)
                                             : 0u;
                    }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float f = a.scale_log2 * k_scale;
                if constexpr (F8 && D::id == AR_DT_BF16) {
                    // The codes are exact in fp16; bf16 queries are once each head is taken
                    // times a power of two that brings its largest element to 2^14 .. 2^15:
                    // what is below 2^-24 then is 2^-38 of the largest.
                    float big = 0.0f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float2 x = unpack2<Bf16>(q[ks][n][half]);
                            big = fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y)));
                        }
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    // the exponents' fields: 2^(141 - e) brings e to 14; within what fp32 holds
                    const int e = (int)(__float_as_uint(big) >> 23);
                    const int up = e == 0 || e == 255 ? 0 : min(141 - e, 126);
                    const float by = __uint_as_float((uint32_t)(127 + up) << 23);
                    f *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float2 x = unpack2<Bf16>(q[ks][n][half]);
                            q[ks][n][half] = pack2<Fp16>(x.x * by, x.y * by);
                        }
                }
                // of the thread's two columns: head 8 n + 2 t + e is that of lane 4 (2 t + e)
                factor[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);
                factor[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[j][n][e] = 0.0f;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                top[n][0] = top[n][1] = -INFINITY;
                total_w[n][0] = total_w[n][1] = 0.0f;
            }
        }
        // the next copies go where the slice before this one was
        copies_wait<kStages - 2>();
        __syncwarp();
        if (u + kStages - 1 < count)
            send(stage == 0 ? kStages - 1 : stage - 1);
        else
            copies_commit();
        const int x = c.unit * kWarps + warp;
        if (x < c.seen.n) {
            const uint32_t kb = ring + stage * 2 * kTile, vb = kb + kTile;
            const int key0 = (x < c.seen.first ? x : x + c.seen.gap) * SL;
            float s[NK][NB][4];
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[k][n][e] = 0.0f;
            if constexpr (F8) {
                // a 16-byte chunk is 16 elements: 4t and 4t + 1 stand for the product's 2t and 2t + 1, the
                // next two for 2t + 8 and 2t + 9, in the queries as here
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2)
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        uint32_t b[4];
                        ldm4(b, kb + F::at(16 * k + 8 * (lane >> 3 & 1) + (lane & 7), ks + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t f[4] = {
                                e4m3_half2(b[2 * i]), e4m3_half2(b[2 * i + 1]),
                                e4m3_half2(b[2 * i] >> 16), e4m3_half2(b[2 * i + 1] >> 16)};
#pragma unroll
                            for (int n = 0; n < NB; ++n)
                                mma<false>(s[k][n], f, q[ks + i][n][0], q[ks + i][n][1]);
                        }
                    }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        uint32_t f[4];
                        ldm4(f, kb + F::at(16 * k + 8 * (lane >> 3 & 1) + (lane & 7),
                                           2 * ks + (lane >> 4)));
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            mma<F::bf16>(s[k][n], f, q[ks][n][0], q[ks][n][1]);
                    }
            }
            // all of the slice's keys seen?
            const auto sees = [&](int j) {
                return j < c.seen.length && (j >= c.seen.low || j < c.seen.sinks);
            };
            const bool all = key0 + SL <= c.seen.length &&
                             (key0 >= c.seen.low || key0 + SL <= c.seen.sinks);
#pragma unroll
            for (int k = 0; k < 2 * NK; ++k) {
                const bool mine = all || sees(key0 + 8 * k + g);
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& z = s[k >> 1][n][2 * (k & 1) + e];
                        z = mine ? z * factor[n][e] : -INFINITY;
                    }
            }
            // values of keys that are not seen need not be finite, and nothing times NaN is NaN
            if (!all) {
#pragma unroll 1
                for (int r = lane; r < SL; r += 32)
                    if (!sees(key0 + r))
#pragma unroll
                        for (int i = 0; i < F::pitch; i += 16)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             vb + r * F::pitch + i),
                                         "r"(0)
                                         : "memory");
                __syncwarp();
            }
            float used[NB][2], now[NB][2];
            bool moved = false;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = top[n][e];
#pragma unroll
                    for (int k = 0; k < NK; ++k)
                        m = fmaxf(m, fmaxf(s[k][n][e], s[k][n][2 + e]));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    now[n][e] = m;
                    used[n][e] = m == -INFINITY ? 0.0f : m;     // a head that has seen nothing yet
                    moved |= m != top[n][e];
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = exp2_fast(top[n][e] - used[n][e]);
                        total_w[n][e] *= f;
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            o[j][n][e] *= f;
                            o[j][n][2 + e] *= f;
                        }
                        top[n][e] = now[n][e];
                    }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    used[n][e] -= F::up;
            uint32_t p[NK][NB][2];
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[k][n][e] = exp2_fast(s[k][n][e] - used[n][e & 1]);
                        total_w[n][e & 1] += s[k][n][e];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        p[k][n][i] = turned(F::bf16 ? pack2<Bf16>(s[k][n][2 * i], s[k][n][2 * i + 1])
                                                    : pack2<Fp16>(s[k][n][2 * i], s[k][n][2 * i + 1]));
                }
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if constexpr (F8) {
#pragma unroll
                    for (int j = 0; j < KS; j += 2) {
                        uint32_t b[4];
                        ldm4_trans(b, vb + F::at(16 * k + 8 * (lane >> 3 & 1) + (lane & 7),
                                                 j + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t b0 = b[2 * i], b1 = b[2 * i + 1];
                            const uint32_t f[4] = {e4m3_half2(__byte_perm(b0, 0, 0x4420)),
                                                   e4m3_half2(__byte_perm(b0, 0, 0x4431)),
                                                   e4m3_half2(__byte_perm(b1, 0, 0x4420)),
                                                   e4m3_half2(__byte_perm(b1, 0, 0x4431))};
#pragma unroll
                            for (int n = 0; n < NB; ++n)
                                mma<false>(o[j + i][n], f, p[k][n][0], p[k][n][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        uint32_t b[4];
                        ldm4_trans(b, vb + F::at(16 * k + 8 * (lane >> 4) + (lane & 7),
                                                 2 * j + (lane >> 3 & 1)));
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            mma<F::bf16>(o[j][n], b, p[k][n][0], p[k][n][1]);
                    }
                }
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;

        const bool item_ends = c.unit + 1 == c.units;
        if (item_ends || u + 1 == count) {
            // the four warps' sums together
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& l = total_w[n][e];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    if (g == 0) {
                        max_sh[warp][head_of(n, e, t)] = top[n][e];
                        sum_sh[warp][head_of(n, e, t)] = l;
                    }
                }
            __syncthreads();
            float best[NB][2], sum[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = head_of(n, e, t);
                    float m = -INFINITY, l = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        m = fmaxf(m, max_sh[w][h]);
                    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        l += sum_sh[w][h] * exp2_fast(max_sh[w][h] - base);
                    best[n][e] = m - F::up;
                    sum[n][e] = l;
                    const float f = exp2_fast(top[n][e] - base);
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        o[j][n][e] *= f;
                        o[j][n][2 + e] *= f;
                    }
                }
            const auto put = [&](float* to) {
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            to[((j * NB + n) * 4 + e) * 32 + lane] = o[j][n][e];
            };
            const auto add = [&](const float* from) {
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[j][n][e] += from[((j * NB + n) * 4 + e) * 32 + lane];
            };
            constexpr int kBuf = 8 * NB * DP;
            if (warp >= 2)
                put(sums + (warp - 2) * kBuf);
            __syncthreads();
            if (warp < 2)
                add(sums + warp * kBuf);
            if (warp == 1)
                put(sums + kBuf);
            __syncthreads();
            if (warp == 0) {
                add(sums + kBuf);
                if (item_ends && whole_start) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int h = head_of(n, e, t);
                            if (h >= rows)
                                continue;
                            const float l = sum[n][e], inv = l > 0.0f || l != l ? v_scale / l : 0.0f;
                            uint8_t* to = a.out.p + c.seq * a.out.row + (q_head + h) * a.out.head;
#pragma unroll
                            for (int j = 0; j < KS; ++j)
                                store_dims<D, F8>(to, a.c.D, j, g, o[j][n][e] * inv, o[j][n][2 + e] * inv);
                            if (a.lse && g == 0)
                                a.lse[(int64_t)c.seq * a.Hq + q_head + h] = (best[n][e] + log2f(l)) * kLn2;
                        }
                } else {
                    // a piece that begins here is part 1, one that began before part 0
                    uint8_t* to = sp.parts + (int64_t)(2 * block + (whole_start ? 1 : 0)) * part_bytes<DP>();
                    float* stats = reinterpret_cast<float*>(to);
                    if (g == 0) {
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                stats[head_of(n, e, t)] = best[n][e];
                                stats[kRows + head_of(n, e, t)] = sum[n][e];
                            }
                    }
                    put(stats + 2 * kRows);
                    if (whole_start && lane == 0) {
                        // the block that has the item's last unit
                        const long long last = u0 + u + (c.units - 1 - c.unit);
                        const int end = (int)(((last + 1) * blocks - 1) / total);
                        sp.desc[block] = make_int4(end - block + 1, c.seq, c.head, c.tile);
                    }
                }
            }
            fresh = true;
            whole_start = true;
        }
        c.next(a, tiles);
    }
}

// Items that several blocks share.  Block (b, y): the item that begins in block b and ends in a
// later one, a part of its elements; a thread has two elements of a head, and all of its loads
// of kJoinAhead parts in flight.
constexpr int kJoinThreads = 256, kJoinAhead = 8;

template <class D, int DP, bool F8, int NB>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttentionArgs a, Split sp)
{
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_trigger();
    pdl_wait();
    const int4 d = sp.desc[blockIdx.x];
    if (d.x == 0)
        return;
    // registers (j, n, e) and (j, n, e + 2)
    const int which = blockIdx.y * (kJoinThreads / 32) + (tid >> 5);
    const int e = which & 1, n = (which >> 1) % NB, j = (which >> 1) / NB;
    if (j >= DP / 16)
        return;
    const int h = head_of(n, e, t), at = ((j * NB + n) * 4 + e) * 32 + lane;
    float m = -INFINITY, l = 0.0f, f0 = 0.0f, f1 = 0.0f;
    for (int p0 = 0; p0 < d.x; p0 += kJoinAhead) {
        float pm[kJoinAhead], pl[kJoinAhead], v0[kJoinAhead], v1[kJoinAhead];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const int p = p0 + i;
            const int slot = p == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + p);
            const float* s = reinterpret_cast<const float*>(sp.parts + (int64_t)slot * part_bytes<DP>());
            pm[i] = p < d.x ? s[h] : -INFINITY;
            pl[i] = p < d.x ? s[kRows + h] : 0.0f;
            v0[i] = p < d.x ? s[2 * kRows + at] : 0.0f;
            v1[i] = p < d.x ? s[2 * kRows + at + 64] : 0.0f;
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            top = fmaxf(top, pm[i]);
        const float base = top == -INFINITY ? 0.0f : top, f = exp2_fast(m - base);
        l *= f;
        f0 *= f;
        f1 *= f;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const float w = exp2_fast(pm[i] - base);
            l = fmaf(pl[i], w, l);
            f0 = fmaf(v0[i], w, f0);
            f1 = fmaf(v1[i], w, f1);
        }
        m = top;
    }
    if (h >= min(kRows, a.G - d.w * kRows))
        return;
    const int q_head = d.z * a.G + d.w * kRows + h;
    const float v_scale = F8 && a.c.scale ? a.c.scale[1] : 1.0f;
    const float inv = l > 0.0f || l != l ? v_scale / l : 0.0f;
    uint8_t* to = a.out.p + d.y * a.out.row + q_head * a.out.head;
    store_dims<D, F8>(to, a.c.D, j, g, f0 * inv, f1 * inv);
    if (a.lse && g == 0 && j == 0)
        a.lse[(int64_t)d.y * a.Hq + q_head] = (m + log2f(l)) * kLn2;
}

template <class D, int DP, bool F8, int NB>
cudaError_t launch_t(const AttentionArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    constexpr int kSmem = kWarps * Fit<F8, NB>::stages * 2 * kTile + 2 * 8 * NB * DP * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(decode_attention_kernel<D, DP, F8, NB>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess)
        return e;
    const int tiles = (a.G + kRows - 1) / kRows;
    // at most so many units
    constexpr int unit = kWarps * Form<D, DP, F8>::SL;
    const int64_t keys = (int64_t)a.c.max_pages << a.c.page_shift;
    const int64_t items = (int64_t)a.c.S * a.c.heads * tiles, most = ((keys + unit - 1) / unit + 1) * items;
    int blocks = Fit<F8, NB>::blocks * d.sms;
    if (most < blocks)
        blocks = (int)most;
    // The workspace: a line for each block, then its two parts.  Without room for as many blocks as
    // whole items keep busy, or one an SM, items stay whole (one sequence of 131072, 64 / 8 heads: 0.5 MB
    // 568 us, 4 MB 93, 8 MB 85, none 2230; 64 x 800-8000, 32 / 8 heads, 512 items: 269, from 4 MB on 188).
    const int64_t fit = (int64_t)(a.work_bytes / (16 + 2 * part_bytes<DP>()));
    const int busy = blocks < d.sms ? blocks : d.sms;
    Split sp{};
    sp.whole = fit < (items < busy ? items : busy);
    if (!sp.whole) {
        if (fit < blocks)
            blocks = (int)fit;
        sp.desc = reinterpret_cast<int4*>(a.work);
        sp.parts = a.work + 16 * (int64_t)blocks;
    }
    const bool joined = !sp.whole && blocks > 1;
    std::unique_lock<std::mutex> both(launches_with(a.work), std::defer_lock);
    if (joined)
        both.lock();
    e = launch_after(decode_attention_kernel<D, DP, F8, NB>, blocks, kThreads, kSmem, s, a, sp, tiles);
    if (e != cudaSuccess || !joined)
        return e;
    constexpr int kJoinWarps = kJoinThreads / 32;
    return launch_after(join_kernel<D, DP, F8, NB>,
                        dim3(blocks, (DP / 16 * NB * 2 + kJoinWarps - 1) / kJoinWarps), kJoinThreads, 0, s,
                        a, sp);
}

template <class D, bool F8>
cudaError_t launch_d(const AttentionArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    // heads in one or two groups of 8 columns; products of 96 elements where the head has no more (33
    // windows of 1000, heads of 80: 17.2 -> 16.4 us; E4M3, 128 x 2048-4096 of 96: 204 -> 200)
    if (a.c.D <= 64)
        return a.G <= 8 ? launch_t<D, 64, F8, 1>(a, d, s) : launch_t<D, 64, F8, 2>(a, d, s);
    if (a.c.D <= 96)
        return a.G <= 8 ? launch_t<D, 96, F8, 1>(a, d, s) : launch_t<D, 96, F8, 2>(a, d, s);
    return a.G <= 8 ? launch_t<D, 128, F8, 1>(a, d, s) : launch_t<D, 128, F8, 2>(a, d, s);
}

}  // namespace

cudaError_t launch_decode_attention(int dtype, bool e4m3, const AttentionArgs& a, cudaStream_t s)
{
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess)
        return e;
    if (dtype == AR_DT_BF16)
        return e4m3 ? launch_d<Bf16, true>(a, d, s) : launch_d<Bf16, false>(a, d, s);
    return e4m3 ? launch_d<Fp16, true>(a, d, s) : launch_d<Fp16, false>(a, d, s);
}

}  // namespace arf

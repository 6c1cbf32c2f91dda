// Attention of one new token per sequence over the paged cache.
//
// Memory bounds it: every key and value is read once, for all the query heads that
// share it.  Those are the rows of m16n8k16 products (up to 16; scores = Q K^T, sums =
// P V), so the scores leave the products in the layout in which the next ones take
// their weights, and no value of theirs passes through shared memory.  At 8 heads per
// key the arithmetic is 8 operations a byte, 54 T a second at the memory's rate: more
// than the fp32 pipes have left beside the conversions, little for these products;
// the instructions on 128 rows of tensor memory would waste seven eighths of them and
// pay a round trip to it for every tile.
//
// A warp has slices of its own: 4 KB of keys and 4 KB of values, a ring of kStages of
// them filled by asynchronous copies, a running maximum and sum, and its own sums.
// Four warps take the four slices of a unit in turn and meet at the end of a piece.
//
// All units of all sequences and heads are one list; a block takes an equal share of it
// wherever that begins and ends, so uneven lengths leave no block behind.  A block
// holds whole items, and at most two pieces of items that other blocks share: those go
// to the workspace as sums, maximum and total, and join_kernel, launched behind it,
// adds them in the order of the blocks.
#include <limits.h>

#include "ar_internal.h"
#include "attention_internal.h"
#include "matmul_internal.h"
#include "tensor_core.cuh"

namespace arf {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kTile = 4096;             // bytes of keys, and of values, of a slice
constexpr int kRows = 16;               // query heads of an item
constexpr int kBlocksPerSm = 2;
constexpr float kLn2 = 0.693147181f;

struct Split {
    int4* desc;                         // [blocks]: parts, sequence, head and tile
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
__device__ __forceinline__ Seen seen_of(const AttentionArgs& a, int seq)
{
    Seen s;
    s.length = clamp_length(a.c, a.c.lengths[seq]);
    s.low = a.window ? max(0, s.length - a.window) : 0;
    s.sinks = min(a.sinks, s.length);
    s.first = (s.sinks + SL - 1) / SL;
    const int end = (s.length + SL - 1) / SL, from = s.low / SL;
    s.gap = max(0, from - s.first);
    s.n = end - s.gap;
    return s;
}

// A place in the list of units: unit `unit` of `units` of head `head` (with its tile of
// query heads) of sequence `seq`.
template <int SL>
struct Cursor {
    int seq, head, unit, units;
    Seen seen;

    __device__ __forceinline__ void enter(const AttentionArgs& a, int s)
    {
        seq = s;
        seen = seen_of<SL>(a, s);
        units = (seen.n + kWarps - 1) / kWarps;
    }
    // to the next unit; false: there is none
    __device__ __forceinline__ void next(const AttentionArgs& a, int heads)
    {
        if (++unit < units)
            return;
        unit = 0;
        if (++head < heads)
            return;
        head = 0;
        int s = seq;
        do {
            if (++s == a.c.S)           // the end of the list: not used further
                return;
            enter(a, s);
        } while (units == 0);
    }
};

template <class D, int DP, bool F8>
struct Form {
    static constexpr int bytes = F8 ? 1 : 2;            // of an element of the cache
    static constexpr int pitch = DP * bytes;            // of a slice's row
    static constexpr int SL = kTile / pitch;            // keys of a slice
    static constexpr bool bf16 = !F8 && D::id == AR_DT_BF16;    // products' type
    // 16-byte chunk `c` of row r: the 8 rows of a matrix load in different banks
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        return r * pitch + ((pitch == 64 ? c ^ (r >> 1 & 3) : c ^ (r & 7)) << 4);
    }
};

// Copies of one slice of a cursor's unit into a stage, by one warp.
template <class D, int DP, bool F8>
__device__ __forceinline__ void load_slice(const AttentionArgs& a, const Cursor<Form<D, DP, F8>::SL>& c,
                                           int head, int warp, int lane, uint32_t stage)
{
    using F = Form<D, DP, F8>;
    const int x = c.unit * kWarps + warp;
    if (x < c.seen.n) {
        const int key0 = (x < c.seen.first ? x : x + c.seen.gap) * F::SL;
        // the page of 8 keys at a time
        int page = -1;
        const int mine = key0 + 8 * lane;
        if (lane < F::SL / 8 && mine < c.seen.length)
            page = a.c.table[(int64_t)c.seq * a.c.max_pages + (mine >> a.c.page_shift)];
        if (page >= a.c.pages)
            page = -1;
        constexpr int kChunks = F::pitch / 16, kStep = 32 / kChunks;    // rows a step
        const int chunk = lane % kChunks;
        const bool used = chunk * 16 < a.c.D * F::bytes;
        const uint8_t* k = a.c.k + head * a.c.k_head + chunk * 16;
        const uint8_t* v = a.c.v + head * a.c.v_head + chunk * 16;
#pragma unroll
        for (int i = 0; i < kTile / 512; ++i) {
            const int r = i * kStep + lane / kChunks;
            const int p = __shfl_sync(0xffffffffu, page, r >> 3);
            const int in = (key0 + r) & ((1 << a.c.page_shift) - 1);
            const bool there = p >= 0;
            const int64_t pp = there ? p : 0;
            if (used) {
                const uint32_t to = stage + F::at(r, chunk);
                copy16(to, k + pp * a.c.k_page + in * a.c.k_row, there);
                copy16(to + kTile, v + pp * a.c.v_page + in * a.c.v_row, there);
            }
        }
    }
    copies_commit();
}

// Element of the head that register (tile j, e) of a thread's sums belongs to.
template <bool F8>
__device__ __forceinline__ int dim_of(int j, int e, int t)
{
    return F8 ? 16 * (j >> 1) + 4 * t + 2 * (e & 1) + (j & 1) : 8 * j + 2 * t + (e & 1);
}

template <class D>
__device__ __forceinline__ void store_element(uint8_t* p, float f)
{
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack2<D>(f, 0.0f);
}

template <class D, int DP, bool F8>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    decode_attention_kernel(AttentionArgs a, Split sp, int tiles)
{
    using F = Form<D, DP, F8>;
    constexpr int SL = F::SL, NT = SL / 8, KS = DP / 16, NO = DP / 8;
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
    for (int i = DP > a.c.D ? tid : INT_MAX; i < kWarps * kStages * 2 * kTile / 16; i += kThreads)
        reinterpret_cast<uint4*>(dyn)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();

    // this block's share of the list of units, and where it begins
    const int per = (a.c.S + kThreads - 1) / kThreads;
    const int s0 = min(tid * per, a.c.S), s1 = min(s0 + per, a.c.S);
    long long mine = 0;
    for (int s = s0; s < s1; ++s)
        mine += (long long)((seen_of<SL>(a, s).n + kWarps - 1) / kWarps) * heads;
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
        u0 = total * block / blocks;
        u1 = total * (block + 1) / blocks;
    }
    if (sp.whole) {
        // items whose first unit lies in the share
        if (tid < 2)
            where_sh[tid] = total;
        __syncthreads();
        long long at = upto - mine;
        for (int s = s0; s < s1; ++s) {
            const int n = (seen_of<SL>(a, s).n + kWarps - 1) / kWarps;
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
            for (int s = s0; s < s1; ++s) {
                const int n = (seen_of<SL>(a, s).n + kWarps - 1) / kWarps;
                const long long end = at + (long long)n * heads;
                if (u0 < end) {
                    const int in = (int)(u0 - at);
                    begin_sh[0] = s;
                    begin_sh[1] = in / n;
                    begin_sh[2] = in % n;
                    break;
                }
                at = end;
            }
        }
    }
    // sequences without a key
    for (int s = block; s < a.c.S; s += (int)gridDim.x) {
        if (seen_of<SL>(a, s).n > 0)
            continue;
        for (int i = tid; i < a.Hq * (a.c.D / 8); i += kThreads) {
            const int h = i / (a.c.D / 8), c = i % (a.c.D / 8);
            *reinterpret_cast<uint4*>(a.out.p + s * a.out.row + h * a.out.head + 16 * c) =
                make_uint4(0, 0, 0, 0);
        }
        if (a.lse)
            for (int h = tid; h < a.Hq; h += kThreads)
                a.lse[(int64_t)s * a.Hq + h] = -INFINITY;
    }
    if (tid == 0 && !sp.whole)
        sp.desc[block] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (u0 >= u1)
        return;

    Cursor<SL> c, ahead;
    c.enter(a, begin_sh[0]);
    c.head = begin_sh[1];
    c.unit = begin_sh[2];
    ahead = c;
    const long long count = u1 - u0;
    float k_scale = 1.0f, v_scale = 1.0f;
    if (F8 && a.c.scale) {
        k_scale = a.c.scale[0];
        v_scale = a.c.scale[1];
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < count) {
            load_slice<D, DP, F8>(a, ahead, ahead.head / tiles, warp, lane, ring + i * 2 * kTile);
            ahead.next(a, heads);
        } else {
            copies_commit();
        }
    }

    uint32_t q[KS][4];
    float o[NO][4];
    float top[2], total_w[2], factor[2];
    bool fresh = true, whole_start = c.unit == 0;
    int stage = 0;
    for (long long u = 0; u < count; ++u) {
        const int head = c.head / tiles, tile = c.head - head * tiles;
        const int rows = min(kRows, a.G - tile * kRows);
        const int q_head = head * a.G + tile * kRows;
        if (fresh) {
            fresh = false;
            const uint8_t* qp = a.q.p + c.seq * a.q.row + q_head * a.q.head;
            const uint8_t* q0 = qp + g * a.q.head;
            const uint8_t* q1 = qp + (g + 8) * a.q.head;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int d = F8 ? 16 * ks + 4 * t + 2 * half : 16 * ks + 8 * half + 2 * t;
                    const bool in = (F8 ? 16 * ks : 16 * ks + 8 * half) < a.c.D;
                    q[ks][2 * half] =
                        in && g < rows ? *reinterpret_cast<const uint32_t*>(q0 + 2 * d) : 0u;
                    q[ks][2 * half + 1] =
                        in && g + 8 < rows ? *reinterpret_cast<const uint32_t*>(q1 + 2 * d) : 0u;
                }
            }
            factor[0] = factor[1] = a.scale_log2 * k_scale;
            if constexpr (F8 && D::id == AR_DT_BF16) {
                // The codes are exact in fp16; bf16 queries are once each row is taken
                // times a power of two that brings its largest element to 2^14 .. 2^15:
                // what is below 2^-24 then is 2^-38 of the largest.
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float big = 0.0f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float2 f = unpack2<Bf16>(q[ks][2 * half + r]);
                            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    // the exponents' fields: 2^(141 - e) brings e to 14; within what fp32 holds
                    const int e = (int)(__float_as_uint(big) >> 23);
                    const int up = e == 0 || e == 255 ? 0 : min(141 - e, 126);
                    const float by = __uint_as_float((uint32_t)(127 + up) << 23);
                    factor[r] *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float2 f = unpack2<Bf16>(q[ks][2 * half + r]);
                            q[ks][2 * half + r] = pack2<Fp16>(f.x * by, f.y * by);
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < NO; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[j][e] = 0.0f;
            top[0] = top[1] = -INFINITY;
            total_w[0] = total_w[1] = 0.0f;
        }
        // the next copies go where the slice before this one was
        copies_wait<kStages - 2>();
        __syncwarp();
        {
            const int to = stage == 0 ? kStages - 1 : stage - 1;
            if (u + kStages - 1 < count) {
                load_slice<D, DP, F8>(a, ahead, ahead.head / tiles, warp, lane, ring + to * 2 * kTile);
                ahead.next(a, heads);
            } else {
                copies_commit();
            }
        }
        const int x = c.unit * kWarps + warp;
        if (x < c.seen.n) {
            const uint32_t kb = ring + stage * 2 * kTile, vb = kb + kTile;
            const int key0 = (x < c.seen.first ? x : x + c.seen.gap) * SL;
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][e] = 0.0f;
            if constexpr (F8) {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 4)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t b[4];
                        ldm4(b, kb + F::at(8 * n + (lane & 7), ks + (lane >> 3)));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma<false>(s[n], q[ks + i], e4m3_half2(b[i]), e4m3_half2(b[i] >> 16));
                    }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        ldm4(b, kb + F::at(8 * n + 8 * (lane >> 4) + (lane & 7),
                                           2 * ks + (lane >> 3 & 1)));
                        mma<F::bf16>(s[n], q[ks], b[0], b[1]);
                        mma<F::bf16>(s[n + 1], q[ks], b[2], b[3]);
                    }
            }
            // all of the slice's keys seen?
            const bool all = key0 + SL <= c.seen.length &&
                             (key0 >= c.seen.low || key0 + SL <= c.seen.sinks);
            uint32_t keep[NT];          // of a pair of keys: which half of a register
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                keep[n] = 0xffffffffu;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][e] *= factor[e >> 1];
                if (!all) {
                    const int j = key0 + 8 * n + 2 * t;
                    const bool k0 = j < c.seen.length && (j >= c.seen.low || j < c.seen.sinks);
                    const bool k1 = j + 1 < c.seen.length &&
                                    (j + 1 >= c.seen.low || j + 1 < c.seen.sinks);
                    keep[n] = (k0 ? 0xffffu : 0u) | (k1 ? 0xffff0000u : 0u);
                    if (!k0)
                        s[n][0] = s[n][2] = -INFINITY;
                    if (!k1)
                        s[n][1] = s[n][3] = -INFINITY;
                }
            }
            float used[2], now[2];
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float m = top[r];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    m = fmaxf(m, fmaxf(s[n][2 * r], s[n][2 * r + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                now[r] = m;
                used[r] = m == -INFINITY ? 0.0f : m;    // a row that has seen nothing yet
                moved |= m != top[r];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = exp2_fast(top[r] - used[r]);
                    total_w[r] *= f;
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        o[j][2 * r] *= f;
                        o[j][2 * r + 1] *= f;
                    }
                    top[r] = now[r];
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = exp2_fast(s[n][e] - used[e >> 1]);
                    total_w[e >> 1] += s[n][e];
                }
#pragma unroll
            for (int kk = 0; kk < NT; kk += 2) {
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* f = &s[kk + (i >> 1)][2 * (i & 1)];
                    p[i] = F::bf16 ? pack2<Bf16>(f[0], f[1]) : pack2<Fp16>(f[0], f[1]);
                }
                if constexpr (F8) {
#pragma unroll
                    for (int j = 0; j < DP / 16; j += 2) {
                        uint32_t b[4];
                        ldm4_trans(b, vb + F::at(8 * kk + 8 * (lane >> 3 & 1) + (lane & 7),
                                                 j + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t b0 = b[2 * i] & keep[kk], b1 = b[2 * i + 1] & keep[kk + 1];
                            mma<false>(o[2 * (j + i)], p, e4m3_half2(__byte_perm(b0, 0, 0x4420)),
                                       e4m3_half2(__byte_perm(b1, 0, 0x4420)));
                            mma<false>(o[2 * (j + i) + 1], p, e4m3_half2(__byte_perm(b0, 0, 0x4431)),
                                       e4m3_half2(__byte_perm(b1, 0, 0x4431)));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < NO; j += 2) {
                        uint32_t b[4];
                        ldm4_trans(b, vb + F::at(8 * kk + 8 * (lane >> 3 & 1) + (lane & 7),
                                                 j + (lane >> 4)));
                        mma<F::bf16>(o[j], p, b[0] & keep[kk], b[1] & keep[kk + 1]);
                        mma<F::bf16>(o[j + 1], p, b[2] & keep[kk], b[3] & keep[kk + 1]);
                    }
                }
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;

        const bool item_ends = c.unit + 1 == c.units;
        if (item_ends || u + 1 == count) {
            // the four warps' sums together
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                total_w[r] += __shfl_xor_sync(0xffffffffu, total_w[r], 1);
                total_w[r] += __shfl_xor_sync(0xffffffffu, total_w[r], 2);
                if (t == 0) {
                    max_sh[warp][g + 8 * r] = top[r];
                    sum_sh[warp][g + 8 * r] = total_w[r];
                }
            }
            __syncthreads();
            float best[2], sum[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                best[r] = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    best[r] = fmaxf(best[r], max_sh[w][g + 8 * r]);
                const float base = best[r] == -INFINITY ? 0.0f : best[r];
                sum[r] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    sum[r] += sum_sh[w][g + 8 * r] * exp2_fast(max_sh[w][g + 8 * r] - base);
                const float f = exp2_fast(top[r] - base);
#pragma unroll
                for (int j = 0; j < NO; ++j) {
                    o[j][2 * r] *= f;
                    o[j][2 * r + 1] *= f;
                }
            }
            const auto put = [&](float* to) {
#pragma unroll
                for (int j = 0; j < NO; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        to[(4 * j + e) * 32 + lane] = o[j][e];
            };
            const auto add = [&](const float* from) {
#pragma unroll
                for (int j = 0; j < NO; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[j][e] += from[(4 * j + e) * 32 + lane];
            };
            constexpr int kBuf = kRows * DP;
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
                    for (int r = 0; r < 2; ++r) {
                        const int row = g + 8 * r;
                        if (row >= rows)
                            continue;
                        const float inv = sum[r] > 0.0f || sum[r] != sum[r] ? v_scale / sum[r] : 0.0f;
                        uint8_t* to = a.out.p + c.seq * a.out.row + (q_head + row) * a.out.head;
#pragma unroll
                        for (int j = 0; j < NO; ++j) {
                            const int d0 = dim_of<F8>(j, 0, t), d1 = dim_of<F8>(j, 1, t);
                            if (d0 >= a.c.D)
                                continue;
                            const float f0 = o[j][2 * r] * inv, f1 = o[j][2 * r + 1] * inv;
                            if constexpr (F8) {
                                store_element<D>(to + 2 * d0, f0);
                                store_element<D>(to + 2 * d1, f1);
                            } else {
                                *reinterpret_cast<uint32_t*>(to + 2 * d0) = pack2<D>(f0, f1);
                            }
                        }
                        if (a.lse && t == 0)
                            a.lse[(int64_t)c.seq * a.Hq + q_head + row] =
                                (best[r] + log2f(sum[r])) * kLn2;
                    }
                } else {
                    // a piece that begins here is part 1, one that began before part 0
                    uint8_t* to = sp.parts + (int64_t)(2 * block + (whole_start ? 1 : 0)) * part_bytes<DP>();
                    float* stats = reinterpret_cast<float*>(to);
                    if (t == 0) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            stats[g + 8 * r] = best[r];
                            stats[kRows + g + 8 * r] = sum[r];
                        }
                    }
                    put(stats + 2 * kRows);
                    if (whole_start && lane == 0) {
                        // the block that has the item's last unit
                        const long long last = u0 + u + (c.units - 1 - c.unit);
                        const int end = (int)(((last + 1) * blocks - 1) / total);
                        sp.desc[block] = make_int4(end - block + 1, c.seq, c.head, 0);
                    }
                }
            }
            fresh = true;
            whole_start = true;
        }
        c.next(a, heads);
    }
}

// Items that several blocks share.  Block (b, y): the item that begins in block b and
// ends in a later one, a quarter of its elements; a warp has a few registers of the
// fragments, each lane one row of them.
constexpr int kJoinThreads = 256, kJoinY = 4, kJoinParts = 32;

template <class D, int DP, bool F8>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttentionArgs a, Split sp, int tiles)
{
    constexpr int kEach = DP / 2 / (kJoinY * kJoinThreads / 32);      // registers of a warp: 2 or 1
    __shared__ float weight[kJoinParts][kRows], max_sh[kRows], sum_sh[kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int4 d = sp.desc[blockIdx.x];
    if (d.x == 0)
        return;
    const auto part = [&](int p) {
        const int slot = p == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + p);
        return reinterpret_cast<const float*>(sp.parts + (int64_t)slot * part_bytes<DP>());
    };
    // maximum and total of each row, 16 threads a row
    {
        const int row = tid >> 4, i = tid & 15;
        float m = -INFINITY, l = 0.0f;
        for (int p = i; p < d.x; p += 16) {
            const float* s = part(p);
            const float pm = s[row], pl = s[kRows + row];
            const float top = fmaxf(m, pm), base = top == -INFINITY ? 0.0f : top;
            l = l * exp2_fast(m - base) + pl * exp2_fast(pm - base);
            m = top;
        }
#pragma unroll
        for (int k = 1; k < 16; k <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, k), ol = __shfl_xor_sync(0xffffffffu, l, k);
            const float top = fmaxf(m, om), base = top == -INFINITY ? 0.0f : top;
            l = l * exp2_fast(m - base) + ol * exp2_fast(om - base);
            m = top;
        }
        if (i == 0) {
            max_sh[row] = m;
            sum_sh[row] = l;
        }
    }
    const int first = (blockIdx.y * (kJoinThreads / 32) + warp) * kEach;     // register 4 j + e
    const int row = (lane >> 2) + 8 * (first >> 1 & 1), t = lane & 3;
    float acc[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        acc[i] = 0.0f;
    for (int p0 = 0; p0 < d.x; p0 += kJoinParts) {
        __syncthreads();
        for (int i = tid; i < kJoinParts * kRows; i += kJoinThreads) {
            const int p = p0 + i / kRows, r = i % kRows;
            const float base = max_sh[r] == -INFINITY ? 0.0f : max_sh[r];
            weight[i / kRows][r] = p < d.x ? exp2_fast(part(p)[r] - base) : 0.0f;
        }
        __syncthreads();
        const int n = min(kJoinParts, d.x - p0);
#pragma unroll 8
        for (int p = 0; p < n; ++p) {
            const float* s = part(p0 + p) + 2 * kRows + first * 32 + lane;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                acc[i] = fmaf(s[32 * i], weight[p][row], acc[i]);
        }
    }
    const int head = d.z / tiles, tile = d.z - head * tiles;
    if (row >= min(kRows, a.G - tile * kRows))
        return;
    const int q_head = head * a.G + tile * kRows + row;
    const float sum = sum_sh[row], v_scale = F8 && a.c.scale ? a.c.scale[1] : 1.0f;
    const float inv = sum > 0.0f || sum != sum ? v_scale / sum : 0.0f;
    uint8_t* to = a.out.p + d.y * a.out.row + q_head * a.out.head;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = dim_of<F8>((first + i) >> 2, (first + i) & 3, t);
        if (at < a.c.D)
            store_element<D>(to + 2 * at, acc[i] * inv);
    }
    if (a.lse && t == 0 && (first & ~3) == 0 && (first & 1) == 0)
        a.lse[(int64_t)d.y * a.Hq + q_head] = (max_sh[row] + log2f(sum)) * kLn2;
}

template <class D, int DP, bool F8>
cudaError_t launch_t(const AttentionArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    constexpr int kSmem = kWarps * kStages * 2 * kTile + 2 * kRows * DP * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(decode_attention_kernel<D, DP, F8>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess)
        return e;
    const int tiles = (a.G + kRows - 1) / kRows;
    // at most so many units
    constexpr int unit = kWarps * Form<D, DP, F8>::SL;
    const int64_t keys = (int64_t)a.c.max_pages << a.c.page_shift;
    const int64_t most = ((keys + unit - 1) / unit) * a.c.S * a.c.heads * tiles;
    int blocks = kBlocksPerSm * d.sms;
    if (most < blocks)
        blocks = (int)most;
    // the workspace: a line for each block, then its two parts
    const int64_t fit = (int64_t)(a.work_bytes / (16 + 2 * part_bytes<DP>()));
    Split sp{};
    sp.whole = fit < (blocks < d.sms ? blocks : d.sms);
    if (!sp.whole) {
        if (fit < blocks)
            blocks = (int)fit;
        sp.desc = reinterpret_cast<int4*>(a.work);
        sp.parts = a.work + 16 * (int64_t)blocks;
    }
    e = launch_after(decode_attention_kernel<D, DP, F8>, blocks, kThreads, kSmem, s, a, sp, tiles);
    if (e != cudaSuccess || sp.whole || blocks == 1)
        return e;
    return launch_after(join_kernel<D, DP, F8>, dim3(blocks, kJoinY), kJoinThreads, 0, s, a, sp, tiles);
}

template <class D, bool F8>
cudaError_t launch_d(const AttentionArgs& a, const DeviceInfo& d, cudaStream_t s)
{
    return a.c.D <= 64 ? launch_t<D, 64, F8>(a, d, s) : launch_t<D, 128, F8>(a, d, s);
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

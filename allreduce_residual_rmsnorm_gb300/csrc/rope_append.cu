// Rotation of the new queries and keys by position, and the keys and values into
// the paged cache.
//
// A block has one row (token).  Its pairs' cosines and sines are computed once, in
// shared memory, and serve all of its heads; a thread turns 16 elements at a time,
// so that both halves of 8 pairs are in its registers.  Every element is read once
// and written once.  The row's place (its sequence, length and page) is a chain of
// three loads, and the elements do not wait for it: the first kAhead pieces of
// every thread are loaded before it.  What bounds it is memory and the latency of that chain (8
// rows on an SM at a time): 4 x 2048 rows of 32 + 8 + 8 heads 36.3 us, 5.5 TB/s (stores without
// the streaming hint 4% more, 7 blocks on an SM 5%, blocks of 64, 96, 192 and 256 threads 17, 2,
// 7 and 40%); 64 rows of 8 + 1 + 1 heads 2.1, a launch.
#include "ar_internal.h"
#include "attention_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kThreads = 128;
constexpr int kMostAhead = 3;   // pieces of 16 elements in flight per thread (16 to 48 bytes spill)

// The division of a piece's number by the pieces of a head, as a multiplication: exact below
// 2^32 / per, and there are below 2^28 pieces of at most 16 a head.
struct Heads {
    unsigned per, inverse;      // inverse: 2^32 / per, rounded up (0: per is 1)
    __device__ __forceinline__ unsigned of(unsigned i) const
    {
        return inverse ? __umulhi(i, inverse) : i;
    }
};

// cos and sin of an angle (half_turns: off by 2^-25 of half a turn at any position, where the
// product in 32 bits is off by position * 2^-24).  A frequency that is not finite gives NaN.
__device__ __forceinline__ float2 turn(int position, float f)
{
    float2 r;
    sincospif(half_turns(position, turns_of(f)) + (f - f), &r.y, &r.x);
    return r;
}

struct Piece {
    const uint8_t* from;        // NULL: none
    int kind, head, first, second;      // kind 0: q, 1: k, 2: v; vectors of 8, second -1: none
    int pair;                   // first pair of the half form, -1: neighbours or a copy
};

template <class D, bool F8, int kAhead>
__global__ void __launch_bounds__(kThreads, kAhead == kMostAhead ? 8 : 0)
    rope_append_kernel(RopeArgs a, Heads turning, Heads copying)
{
    __shared__ __align__(16) float2 cs[AR_MAX_HEAD_DIM / 2];
    __shared__ int found, place[2];
    const int row = blockIdx.x, tid = threadIdx.x;
    if (tid == 0)
        found = 0;
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    // pieces of a rotated head (the pairs of the half form, then the rest) and of a copied one
    const int half = a.interleaved ? 0 : a.rot / 16;
    const int rest = half * 2;
    const unsigned vecs = a.c.D / 8;
    const unsigned turned = (a.Hq + a.c.heads) * turning.per, total = turned + a.c.heads * copying.per;

    const auto piece = [&](unsigned i) {
        Piece p;
        p.pair = -1;
        unsigned in;
        if (i < turned) {
            const unsigned h = turning.of(i);
            in = i - h * turning.per;
            p.kind = h < (unsigned)a.Hq ? 0 : 1;
            p.head = p.kind ? h - a.Hq : h;
            if (in < (unsigned)half) {
                p.pair = 8 * in;
                p.first = in;
                p.second = in + half;
            } else {
                p.first = rest + 2 * (in - half);
            }
        } else {
            const unsigned h = copying.of(i - turned);
            in = i - turned - h * copying.per;
            p.kind = 2;
            p.head = h;
            p.first = 2 * in;
        }
        if (p.pair < 0)
            p.second = p.first + 1 < (int)vecs ? p.first + 1 : -1;
        const Rows& r = p.kind == 0 ? a.q : p.kind == 1 ? a.k : a.v;
        p.from = i < total ? r.p + row * r.row + p.head * r.head : nullptr;
        return p;
    };

    // The row's sequence: the thread that sees it has the length, too, and finds the page.
    uint4 x[kAhead][2];
    Piece pieces[kAhead];
    int lo = 0, hi = 0, length = 0;
    if (tid < a.c.S && a.starts) {
        lo = a.starts[tid];
        hi = a.starts[tid + 1];
        length = a.c.lengths[tid];
    }
    // what the turns need beside the place
    float freq = 0.0f, inverse[2] = {1.0f, 1.0f};
    int where = 0;
    if (tid < a.rot / 2) {
        freq = a.inv_freq[tid];
        if (a.positions) {
            int axis = 0;
            while (tid >= a.ends[axis])     // ends[axes - 1] is rot / 2
                ++axis;
            where = a.positions[(int64_t)axis * a.T + row];
        }
    }
    if (F8 && a.c.scale) {
        inverse[0] = a.c.scale[0];
        inverse[1] = a.c.scale[1];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const Piece p = pieces[j] = piece(tid + j * kThreads);
        if (p.from) {
            x[j][0] = ld_stream(p.from + 16 * p.first);
            if (p.second >= 0)
                x[j][1] = ld_stream(p.from + 16 * p.second);
        }
    }
    const auto page_of = [&](int seq, int at) {
        return at < 0 ? -1 : a.c.table[(int64_t)seq * a.c.max_pages + (at >> a.c.page_shift)];
    };
    int index, page;
    if (a.starts) {
        bool falls = false;
        for (int s = tid; s < a.c.S; s += kThreads) {
            if (s >= kThreads) {
                lo = a.starts[s];
                hi = a.starts[s + 1];
                length = a.c.lengths[s];
            }
            falls |= lo > hi;
            // one sequence has the row, unless the starts decrease: then none has any
            if (lo >= 0 && lo <= row && row < hi && hi <= a.T && atomicExch(&found, 1) == 0) {
                place[0] = clamp_length(a.c, length) - (hi - row);
                place[1] = page_of(s, place[0]);
            }
        }
        if (__syncthreads_or(falls) || !found)
            return;
        index = place[0];
        page = place[1];
    } else {
        index = clamp_length(a.c, a.c.lengths[row]) - 1;
        page = page_of(row, index);
    }
    const bool placed = page >= 0 && page < a.c.pages;
    const int in_page = index & ((1 << a.c.page_shift) - 1);
    if (tid < a.rot / 2)
        cs[tid] = turn(a.positions ? where : index, freq);
    inverse[0] = 1.0f / inverse[0];
    inverse[1] = 1.0f / inverse[1];
    __syncthreads();

    const auto finish = [&](const Piece& p, const uint4& x0, const uint4& x1) {
        if (p.kind && !placed)
            return;
        float f[2][8];
        unpack8<D>(x0, f[0]);
        if (p.second >= 0)
            unpack8<D>(x1, f[1]);
        if (p.pair >= 0) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {        // two pairs' cosines and sines a load
                const float4 c = *reinterpret_cast<const float4*>(&cs[p.pair + e]);
                const float u0 = f[0][e], w0 = f[1][e], u1 = f[0][e + 1], w1 = f[1][e + 1];
                f[0][e] = fmaf(u0, c.x, -(w0 * c.y));
                f[1][e] = fmaf(w0, c.x, u0 * c.y);
                f[0][e + 1] = fmaf(u1, c.z, -(w1 * c.w));
                f[1][e + 1] = fmaf(w1, c.z, u1 * c.w);
            }
        } else if (a.interleaved && p.kind < 2) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int first = (p.first + v) * 8;
                if (first < a.rot) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 c = cs[first / 2 + e];
                        const float u = f[v][2 * e], w = f[v][2 * e + 1];
                        f[v][2 * e] = fmaf(u, c.x, -(w * c.y));
                        f[v][2 * e + 1] = fmaf(w, c.x, u * c.y);
                    }
                }
            }
        }
        uint8_t* to;
        if (p.kind == 0)
            to = a.q_out.p + row * a.q_out.row + p.head * a.q_out.head;
        else if (p.kind == 1)
            to = a.c.k + page * a.c.k_page + in_page * a.c.k_row + p.head * a.c.k_head;
        else
            to = a.c.v + page * a.c.v_page + in_page * a.c.v_row + p.head * a.c.v_head;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = v ? p.second : p.first;
            if (at < 0)
                continue;
            if (F8 && p.kind) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[v][e] *= inverse[p.kind - 1];
                *reinterpret_cast<uint2*>(to + 8 * at) = e4m3x8(f[v]);
            } else {
                __stcs(reinterpret_cast<uint4*>(to + 16 * at), pack8<D>(f[v]));
            }
        }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        if (pieces[j].from)
            finish(pieces[j], x[j][0], x[j][1]);
    }
    for (unsigned i = tid + kAhead * kThreads; i < total; i += kThreads) {
        const Piece p = piece(i);
        uint4 x0 = ld_stream(p.from + 16 * p.first), x1 = x0;
        if (p.second >= 0)
            x1 = ld_stream(p.from + 16 * p.second);
        finish(p, x0, x1);
    }
}

Heads heads_of(unsigned per)
{
    return Heads{per, per == 1 ? 0u : (unsigned)(((1ull << 32) + per - 1) / per)};
}

// As many pieces ahead as the row gives a thread: those that are not there cost as much as the
// others (7.2 instead of 4.0 us at 1479 rows of 15 + 5 + 5 heads of 80).
template <class D, bool F8>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t s)
{
    const unsigned half = a.interleaved ? 0 : a.rot / 16, vecs = a.c.D / 8;
    const Heads turning = heads_of(half + (vecs - 2 * half + 1) / 2), copying = heads_of((vecs + 1) / 2);
    const uint64_t pieces = ((uint64_t)a.Hq + a.c.heads) * turning.per + (uint64_t)a.c.heads * copying.per;
    if (pieces <= kThreads)
        return launch_after(rope_append_kernel<D, F8, 1>, a.T, kThreads, 0, s, a, turning, copying);
    if (pieces <= 2 * kThreads)
        return launch_after(rope_append_kernel<D, F8, 2>, a.T, kThreads, 0, s, a, turning, copying);
    return launch_after(rope_append_kernel<D, F8, kMostAhead>, a.T, kThreads, 0, s, a, turning, copying);
}

}  // namespace

cudaError_t launch_rope_append(int dtype, bool e4m3, const RopeArgs& a, cudaStream_t s)
{
    if (dtype == AR_DT_BF16)
        return e4m3 ? launch_t<Bf16, true>(a, s) : launch_t<Bf16, false>(a, s);
    return e4m3 ? launch_t<Fp16, true>(a, s) : launch_t<Fp16, false>(a, s);
}

}  // namespace arf

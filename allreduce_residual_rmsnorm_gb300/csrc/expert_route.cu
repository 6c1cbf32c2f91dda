// Routing to experts: scores, groups, top-k and weights of one token row per
// warp.  Expert e = lane + 32 i starts in register i of its lane; each lane
// sorts its own, and a pick is the largest of the 32 heads.  Bounded by its
// instructions, 1570 a row with 256 sigmoid scores, a bias, 8 groups and 8 chosen
// (8192 rows: 15.1 us; their 9 MB are 1.4 us of memory time).
//
// The order of the choice values c = s + bias is that of the real numbers.
// Without a bias, or with the same one everywhere, it is the order of the
// logits, and no score is compared at all.  Otherwise c is computed in fp32
// with a known error bound, and a row where a pick's runner-up, or a group's,
// lies within that bound is decided again in fp64 for the values within it.
// fp64 runs at 1/64 of the fp32 rate here, so deciding everything in fp64 would
// take longer than the whole kernel; a border that close comes up in about one
// row of 300 (256 sigmoid scores, 8 chosen).
//
// Error bound, relative to the largest score, with u = 2^-24: __expf is off by
// (2 + 1.17 |x|) 2u of its value, which moves a sigmoid by s (1 - s) of that,
// below 0.76 * 2u; 1 + e is off by u, __fdividef by 4u: below 1.7 * 2^-22 in
// all.  Softmax also has the fp32 sum of up to 32 values a lane and 5 butterfly
// steps, below 2^-18.4.  c itself is rounded once, u |c|.  Two values compared:
// twice that.
#include <math.h>

#include "expert_internal.h"
#include "expert_vec.cuh"

namespace arf {
namespace {

constexpr int kWarps = 4;       // rows per block

// Order-preserving map of floats to unsigned: 0 is kept for "out", NaN is 1,
// below every number.  -0 counts as +0.
__device__ __forceinline__ uint32_t to_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return v == v ? k : 1u;
}
__device__ __forceinline__ float from_key(uint32_t k)
{
    const uint32_t u = k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u);
    return __uint_as_float(k == 1u ? 0x7fc00000u : u);
}

// a call's sizes, divided out on the host: experts per group, lanes per group and
// their logarithm, 1 / experts per group
struct Shape {
    int size, team, shift;
    float inv_size;
};

struct Row {
    int softmax;
    float max, inv_sum;         // softmax: row maximum, 1 / sum of exponentials
    double sum;                 // the sum in fp64, once it was needed (else 0)
};

__device__ __forceinline__ float score_of(const Row& r, float x)
{
    return r.softmax ? expf(x - r.max) * r.inv_sum : 1.0f / (1.0f + expf(-x));
}

// the same with the fast exponential and division, for the order
__device__ __forceinline__ float quick_score(const Row& r, float x)
{
    return r.softmax ? __expf(x - r.max) * r.inv_sum : __fdividef(1.0f, 1.0f + __expf(-x));
}

// the choice value in fp64
__device__ __noinline__ double exact_choice(int softmax, float max, double sum, float x, float b)
{
    const double s = softmax ? exp((double)x - (double)max) / sum : 1.0 / (1.0 + exp(-(double)x));
    return s + (double)b;
}

// the softmax sum in fp64: once per row, where a border needs it
template <class D>
__device__ __noinline__ double exact_sum(const void* logits, const float* bias, uint64_t at, int E,
                                         float max, int lane)
{
    double z = 0.0;
    for (int e = lane; e < E; e += 32) {
        const float x = load1<D>(logits, at + e);
        if (x != -INFINITY && !(bias && bias[e] == -INFINITY))
            z += exp((double)x - (double)max);
    }
    for (int m = 16; m >= 1; m >>= 1)
        z += __shfl_xor_sync(0xffffffffu, z, m);
    return z;
}

// Groups that stay, as a mask over lanes: group g is bit g * team.  `key` holds
// the row's ordering values as keys (0: out).
template <class D>
__device__ __forceinline__ uint32_t kept_groups(const RouteArgs& a, Row& r, const uint32_t* key,
                                                uint64_t at, bool by_logit, float bias0,
                                                float base_err, int lane, const Shape& sh)
{
    const uint32_t full = 0xffffffffu;
    const int size = sh.size, team = sh.team;
    const int g = lane >> sh.shift, sub = lane & (team - 1);
    uint32_t k1 = 0, k2 = 0;
    if (g < a.G) {
        // each team starts at a place of its own: with 32 experts a group they
        // would all read the same bank
        const int n = (size - sub + team - 1) >> sh.shift;
        int t = sub + (g < n ? g * team : 0);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const uint32_t k = key[g * size + t];
            k2 = max(k2, min(k1, k));
            k1 = max(k1, k);
            t += team;
            t = t < size ? t : sub;
        }
    }
    for (int m = team >> 1; m >= 1; m >>= 1) {
        const uint32_t o1 = __shfl_xor_sync(full, k1, m), o2 = __shfl_xor_sync(full, k2, m);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
    }
    const bool top2 = a.group_score == AR_GROUP_TOP2;
    uint32_t gk = k1;
    float err = 0.0f;
    if (k1 != 0 && (top2 || !by_logit)) {
        const float v1 = by_logit ? quick_score(r, from_key(k1)) + bias0 : from_key(k1);
        const float v2 = !top2 || k2 == 0 ? 0.0f
                         : by_logit       ? quick_score(r, from_key(k2)) + bias0
                                          : from_key(k2);
        gk = to_key(v1 + v2);
        err = base_err + 0x1p-22f * (fabsf(v1) + fabsf(v2));
        if (!(err < INFINITY))
            err = 0.0f;
    }
    const auto rank_among = [&](auto mine) {
        int rank = 0;
        for (int o = 0; o < a.G; ++o) {
            const auto v = __shfl_sync(full, mine, o << sh.shift);
            rank += v > mine || (v == mine && o < g);
        }
        return rank;
    };
    bool kept = (rank_among(gk) < a.keep) & (g < a.G);
    // decided, unless the least value that a kept group may have is not above
    // the largest that a dropped one may have
    if (top2 || !by_logit) {
        const float v = from_key(gk);
        const uint32_t low = gk > 1 ? to_key(v - err) : gk, high = gk > 1 ? to_key(v + err) : gk;
        const uint32_t least = __reduce_min_sync(full, kept ? low : full);
        const uint32_t most = __reduce_max_sync(full, !kept && g < a.G ? high : 0u);
        if (least <= most && most > 1) {
            if (r.softmax && r.sum == 0.0)
                r.sum = exact_sum<D>(a.logits, a.bias, at, a.E, r.max, lane);
            // the values that can be among the largest (two) of their group
            const uint32_t last = top2 && k2 > 1 ? k2 : k1;
            const uint32_t from = by_logit ? last : max(2u, to_key(from_key(last) - 2.0f * err));
            double d1 = -INFINITY, d2 = -INFINITY;
            const auto weigh = [&](int e) {
                const double c = exact_choice(r.softmax, r.max, r.sum,
                                              load1<D>(a.logits, at + e),
                                              a.bias ? a.bias[e] : 0.0f);
                d2 = fmax(d2, fmin(d1, c));
                d1 = fmax(d1, c);
            };
            // found first, then weighed together: fp64 is slow, and the lanes
            // find theirs in different steps
            int hits = 0, h0 = 0, h1 = 0;
            if (g < a.G && gk > 1) {
                for (int t = sub; t < size; t += team) {
                    const int e = g * size + t;
                    if (key[e] >= from) {
                        h1 = hits == 1 ? e : h1;
                        h0 = hits == 0 ? e : h0;
                        if (++hits > 2)
                            weigh(e);
                    }
                }
            }
            if (hits > 0)
                weigh(h0);
            if (hits > 1)
                weigh(h1);
            __syncwarp();
            for (int m = team >> 1; m >= 1; m >>= 1) {
                const double o1 = __shfl_xor_sync(full, d1, m), o2 = __shfl_xor_sync(full, d2, m);
                d2 = fmax(fmin(d1, o1), fmax(d2, o2));
                d1 = fmax(d1, o1);
            }
            const double none = gk == 1 ? -1.7e308 : -INFINITY;
            const double d = gk <= 1 ? none : top2 && k2 > 1 ? d1 + d2 : d1;
            kept = (rank_among(d) < a.keep) & (g < a.G);
        }
    }
    return __ballot_sync(full, kept);
}

// The picks of a row with a border within the error bound: values within it of
// the largest left are compared in fp64.  Returns lane j's pick, or -1.  Reads
// the row again for each pick: rare, and small beside the registers that
// keeping everything would cost the common path.
template <class D>
__device__ __noinline__ int exact_picks(const RouteArgs& a, const Row& r0, uint64_t at,
                                        uint32_t kept, const Shape& sh, float base_err, int lane)
{
    const uint32_t full = 0xffffffffu;
    Row r = r0;
    if (r.softmax && r.sum == 0.0)
        r.sum = exact_sum<D>(a.logits, a.bias, at, a.E, r.max, lane);
    uint32_t taken = 0;         // bit i: expert lane + 32 i
    const auto key_of = [&](int e) {
        const float x = load1<D>(a.logits, at + e), b = a.bias[e];
        const bool out = x == -INFINITY || b == -INFINITY || (taken >> (e >> 5) & 1u) ||
                         (a.G > 1 &&
                          !(kept >> ((int)(((float)e + 0.5f) * sh.inv_size) * sh.team) & 1u));
        return out ? 0u : to_key(quick_score(r, x) + b);
    };
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        uint32_t lb = 0;
        for (int e = lane; e < a.E; e += 32)
            lb = max(lb, key_of(e));
        const uint32_t best = __reduce_max_sync(full, lb);
        if (best == 0)
            break;
        uint32_t thr = best;
        if (best > 1) {
            const float v = from_key(best), low = v - (base_err + 0x1p-22f * fabsf(v));
            thr = low > -INFINITY ? to_key(low) : best;
        }
        double c = -INFINITY;
        int pick = INT_MAX;
        for (int e = lane; e < a.E; e += 32) {
            if (key_of(e) < thr)
                continue;
            const double v = best == 1 ? 0.0
                                       : exact_choice(r.softmax, r.max, r.sum,
                                                      load1<D>(a.logits, at + e), a.bias[e]);
            if (pick == INT_MAX || v > c) {
                c = v;
                pick = e;
            }
        }
        for (int m = 16; m >= 1; m >>= 1) {
            const double oc = __shfl_xor_sync(full, c, m);
            const int op = __shfl_xor_sync(full, pick, m);
            if (op != INT_MAX && (pick == INT_MAX || oc > c || (oc == c && op < pick))) {
                c = oc;
                pick = op;
            }
        }
        if (lane == j)
            mine = pick;
        if ((pick & 31) == lane)
            taken |= 1u << (pick >> 5);
    }
    return mine;
}

// Descending order of a lane's values: Batcher's odd-even merge sort, written as
// templates so that every index is a constant and the values stay in registers.
template <int A, int B, int V>
__device__ __forceinline__ void larger_first(uint64_t (&v)[V])
{
    const uint64_t a = v[A], b = v[B];
    v[A] = a > b ? a : b;
    v[B] = a > b ? b : a;
}
template <int I, int R, int END, int V>
__device__ __forceinline__ void larger_first_from(uint64_t (&v)[V])
{
    if constexpr (I + R < END) {
        larger_first<I, I + R>(v);
        larger_first_from<I + 2 * R, R, END>(v);
    }
}
template <int LO, int N, int R, int V>
__device__ __forceinline__ void merge_down(uint64_t (&v)[V])
{
    if constexpr (2 * R < N) {
        merge_down<LO, N, 2 * R>(v);
        merge_down<LO + R, N, 2 * R>(v);
        larger_first_from<LO + R, R, LO + N>(v);
    } else {
        larger_first<LO, LO + R>(v);
    }
}
template <int LO, int N, int V>
__device__ __forceinline__ void sort_down(uint64_t (&v)[V])
{
    if constexpr (N > 1) {
        sort_down<LO, N / 2>(v);
        sort_down<LO + N / 2, N / 2>(v);
        merge_down<LO, N, 1>(v);
    }
}

template <class D, int V>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(RouteArgs a, Shape sh)
{
    extern __shared__ uint32_t key_sh[];        // [kWarps][E] with groups
    const uint32_t full = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    pdl_trigger();
    if (t >= a.T)
        return;
    pdl_wait();
    const uint64_t at = (uint64_t)t * a.E;

    // logits (-inf: out) and whether the bias moves the order at all
    float x[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < a.E ? load1<D>(a.logits, at + e) : -INFINITY;
        b[i] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
    bool by_logit = true;
    float bias0 = 0.0f;
    if (a.bias) {
        float blo = INFINITY, bhi = -INFINITY;
        bool bnan = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = b[i] == -INFINITY ? -INFINITY : x[i];
            const bool in = x[i] != -INFINITY;
            blo = in ? fminf(blo, b[i]) : blo;
            bhi = in ? fmaxf(bhi, b[i]) : bhi;
            bnan |= in && b[i] != b[i];
        }
        blo = from_key(__reduce_min_sync(full, to_key(blo)));
        bhi = from_key(__reduce_max_sync(full, to_key(bhi)));
        by_logit = !__any_sync(full, bnan) && blo >= bhi && fabsf(bhi) < INFINITY;
        bias0 = by_logit ? bhi : 0.0f;
    }

    Row r{a.score == AR_SCORE_SOFTMAX, 0.0f, 1.0f, 0.0};
    if (r.softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
            m = fmaxf(m, x[i]);
        r.max = from_key(__reduce_max_sync(full, to_key(m)));
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            z += x[i] == -INFINITY ? 0.0f : expf(x[i] - r.max);
#pragma unroll
        for (int m2 = 16; m2 >= 1; m2 >>= 1)
            z += __shfl_xor_sync(full, z, m2);
        r.inv_sum = 1.0f / z;
    }
    // twice the error bound of a choice value, without its 2^-22 |c|
    const float base_err = r.softmax ? 0x1p-17f * r.inv_sum : 0x1p-20f;

    // keys of the ordering values: logits, or choice values
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float o = by_logit ? x[i] : quick_score(r, x[i]) + b[i];
        key[i] = x[i] == -INFINITY ? 0u : to_key(o);
    }
    uint32_t kept = full;
    if (a.G > 1) {
        uint32_t* keys = key_sh + warp * a.E;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < a.E)
                keys[lane + 32 * i] = key[i];
        __syncwarp();
        kept = kept_groups<D>(a, r, keys, at, by_logit, bias0, base_err, lane, sh);
        if (sh.size % 32 == 0) {
            // a register of all lanes lies in one group
            int left = sh.size, bit = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                key[i] = kept >> (bit & 31) & 1u ? key[i] : 0u;
                left -= 32;
                bit += left == 0 ? sh.team : 0;
                left = left == 0 ? sh.size : left;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // e < 1024: (e + 1/2) / size in fp32 is below the next whole
                // number; an expert behind the last one has key 0 already
                const int g = (int)(((float)(lane + 32 * i) + 0.5f) * sh.inv_size);
                if (!(kept >> (g << sh.shift & 31) & 1u))
                    key[i] = 0u;
            }
        }
    }
    // key, then the lower expert
    uint64_t v[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = (uint64_t)key[i] << 32 | (uint32_t)~(lane + 32 * i);
    sort_down<0, V>(v);

    // Picks in fp32 order, one more than chosen (lane j: the j-th)
    int mine = -1;
    uint32_t my_key = 0;
    const auto take = [&](int j) {
        const uint32_t head = (uint32_t)(v[0] >> 32);
        const uint32_t best = __reduce_max_sync(full, head);
        if (best == 0)
            return false;
        const uint32_t who = __ballot_sync(full, head == best);
        int src = __ffs(who) - 1;
        uint32_t pick = ~__shfl_sync(full, (uint32_t)v[0], src);
        if (who & (who - 1)) {
            pick = __reduce_min_sync(full, head == best ? ~(uint32_t)v[0] : full);
            src = (int)(pick & 31);
        }
        if (lane == j) {
            mine = (int)pick;
            my_key = best;
        }
        if (lane == src) {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i)
                v[i] = v[i + 1];
            v[V - 1] = 0ull;
        }
        return true;
    };
    int picks = 0;
    for (; picks <= min(a.k, 31); ++picks)
        if (!take(picks))
            break;
    if (!by_logit) {
        // a next pick with this key or more is too close to this lane's
        const auto border_of = [&](uint32_t k) {
            const float c = from_key(k), low = c - (base_err + 0x1p-22f * fabsf(c));
            return k > 1 && low > -INFINITY ? to_key(low) : full;
        };
        const uint32_t border = border_of(my_key);
        const uint32_t next = __shfl_down_sync(full, my_key, 1);
        bool close = __any_sync(full, lane < picks - 1 && next >= border);
        if (a.k == 32)          // its runner-up is no pick
            close |= __reduce_max_sync(full, (uint32_t)(v[0] >> 32)) >= __shfl_sync(full, border, 31);
        if (close) {
            // past the last one while the next is too close to it
            uint32_t edge = __shfl_sync(full, border, max(picks - 1, 0)), rest;
            while ((rest = __reduce_max_sync(full, (uint32_t)(v[0] >> 32))) != 0 && rest >= edge &&
                   picks < 32) {
                take(picks++);
                edge = border_of(rest);
            }
            if (picks == 32 && rest >= edge) {
                // 32 picks and no end of close ones: one by one
                mine = exact_picks<D>(a, r, at, kept, sh, base_err, lane);
            } else {
                // every value left is below all of these: order them in fp64
                if (r.softmax && r.sum == 0.0)
                    r.sum = exact_sum<D>(a.logits, a.bias, at, a.E, r.max, lane);
                double c = -INFINITY;       // NaN: behind the numbers
                if (mine >= 0 && my_key > 1)
                    c = exact_choice(r.softmax, r.max, r.sum, load1<D>(a.logits, at + mine),
                                     a.bias[mine]);
                __syncwarp();
                int rank = 0;
                for (int o = 0; o < picks; ++o) {
                    const double oc = __shfl_sync(full, c, o);
                    const int oe = __shfl_sync(full, mine, o);
                    rank += oc > c || (oc == c && oe < mine);
                }
                int sorted = -1;
                for (int o = 0; o < picks; ++o) {
                    const int orank = __shfl_sync(full, rank, o), oe = __shfl_sync(full, mine, o);
                    sorted = orank == lane ? oe : sorted;
                }
                mine = sorted;
            }
        }
    }
    if (lane >= a.k)
        mine = -1;

    // Weights.  Renormalised ones divide out the largest exponential of the
    // chosen first, so that scores below the fp32 range keep their ratios.
    const float xm = mine >= 0 ? load1<D>(a.logits, at + mine) : -INFINITY;
    float s = 0.0f;
    if (!a.renorm) {
        s = mine >= 0 ? score_of(r, xm) : 0.0f;
    } else {
        // sigmoid: s = e^min(x, 0) / (1 + e^-|x|)
        const float low = r.softmax || xm < 0.0f ? xm : 0.0f;
        const float top = from_key(__reduce_max_sync(full, mine >= 0 ? to_key(low) : 0u));
        if (mine >= 0) {
            s = expf(low - top);
            if (!r.softmax)
                s /= 1.0f + expf(-fabsf(xm));
            else if (!(r.inv_sum == r.inv_sum))
                s = r.inv_sum;          // a NaN in the row's sum reaches every weight
        }
        float sum = s;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1)
            sum += __shfl_xor_sync(full, sum, m);
        s = mine >= 0 ? s / sum : 0.0f;
    }
    if (lane < a.k) {
        a.ids[(uint64_t)t * a.k + lane] = mine;
        a.weights[(uint64_t)t * a.k + lane] = s * a.scale;
    }
}

template <class D>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t s)
{
    Shape sh{a.E / a.G, 32, 5, 1.0f / (float)(a.E / a.G)};
    while (sh.team * a.G > 32) {
        sh.team >>= 1;
        --sh.shift;
    }
    const unsigned grid = (unsigned)((a.T - 1) / kWarps + 1);
    const size_t smem = a.G > 1 ? sizeof(uint32_t) * kWarps * a.E : 0;
    const int per_lane = (a.E + 31) / 32;
    if (per_lane <= 1)
        return launch_after(route_kernel<D, 1>, grid, 32 * kWarps, smem, s, a, sh);
    if (per_lane <= 2)
        return launch_after(route_kernel<D, 2>, grid, 32 * kWarps, smem, s, a, sh);
    if (per_lane <= 4)
        return launch_after(route_kernel<D, 4>, grid, 32 * kWarps, smem, s, a, sh);
    if (per_lane <= 8)
        return launch_after(route_kernel<D, 8>, grid, 32 * kWarps, smem, s, a, sh);
    if (per_lane <= 16)
        return launch_after(route_kernel<D, 16>, grid, 32 * kWarps, smem, s, a, sh);
    return launch_after(route_kernel<D, 32>, grid, 32 * kWarps, smem, s, a, sh);
}

}  // namespace

cudaError_t launch_route(int dtype, const RouteArgs& a, cudaStream_t s)
{
    switch (dtype) {
    case AR_DT_BF16: return launch_route_t<Bf16>(a, s);
    case AR_DT_FP16: return launch_route_t<Fp16>(a, s);
    default: return launch_route_t<F32>(a, s);
    }
}

}  // namespace arf

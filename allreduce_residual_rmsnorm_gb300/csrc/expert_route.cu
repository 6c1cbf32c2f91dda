// Routing to experts: scores, groups, top-k and weights of one token row per
// warp.  Expert e = lane + 32 i sits in register i of its lane.
//
// The order of the choice values c = s + bias is that of the real numbers.
// Without a bias, or with the same one everywhere, it is the order of the
// logits, and no score is compared at all.  Otherwise c is computed in fp32
// with a known error bound, and a pick whose runner-up lies within that bound
// is decided again in fp64 for the values within it alone.  fp64 runs at about
// 1/60 of the fp32 rate here, so deciding everything in fp64 would take longer
// than the whole kernel; a border that close comes up in about one row of 300
// (256 sigmoid scores, 8 chosen).
//
// Error bound, relative to the largest score: sigmoid: expf 2^-23 (1 ulp),
// 1 + e and the division 2^-24 each, below 2^-22 in all; softmax also has the
// fp32 sum of up to 32 values a lane and 5 butterfly steps, below 2^-18.8.
// c itself is rounded once, 2^-24 |c|.  Two values compared: twice that.
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
    const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return v == v ? k : 1u;
}
__device__ __forceinline__ float from_key(uint32_t k)
{
    return k == 1u ? __uint_as_float(0x7fc00000u)
                   : __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct Row {
    int softmax;
    float max, inv_sum;         // softmax: row maximum, 1 / sum of exponentials
    double sum;                 // the sum in fp64, once it was needed (else 0)
};

__device__ __forceinline__ float score_of(const Row& r, float x)
{
    return r.softmax ? expf(x - r.max) * r.inv_sum : 1.0f / (1.0f + expf(-x));
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

// Groups that stay, as a mask over lanes: group g is bit g * team.  `choice`
// holds the ordering values of the row (-inf: out).
template <class D>
__device__ __forceinline__ uint32_t kept_groups(const RouteArgs& a, Row& r, const float* choice,
                                                uint64_t at, bool by_logit, float bias0,
                                                float base_err, int lane, int team)
{
    const uint32_t full = 0xffffffffu;
    const int size = a.E / a.G;
    const int g = lane / team, sub = lane & (team - 1);
    uint32_t k1 = 0, k2 = 0;
    if (g < a.G) {
        for (int t = sub; t < size; t += team) {
            const float v = choice[g * size + t];
            const uint32_t k = v == -INFINITY ? 0u : to_key(v);
            k2 = max(k2, min(k1, k));
            k1 = max(k1, k);
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
        const float v1 = by_logit ? score_of(r, from_key(k1)) + bias0 : from_key(k1);
        const float v2 = !top2 || k2 == 0 ? 0.0f
                         : by_logit       ? score_of(r, from_key(k2)) + bias0
                                          : from_key(k2);
        gk = to_key(v1 + v2);
        err = base_err + 0x1p-22f * (fabsf(v1) + fabsf(v2));
        if (!(err < INFINITY))
            err = 0.0f;
    }
    const auto rank_among = [&](auto mine) {
        int rank = 0;
        for (int o = 0; o < a.G; ++o) {
            const auto v = __shfl_sync(full, mine, o * team);
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
            const float cut = from_key(top2 && k2 > 1 ? k2 : k1);
            const uint32_t from = by_logit ? (top2 && k2 > 1 ? k2 : k1)
                                           : max(2u, to_key(cut - 2.0f * err));
            double d1 = -INFINITY, d2 = -INFINITY;
            if (g < a.G && gk > 1) {
                for (int t = sub; t < size; t += team) {
                    const int e = g * size + t;
                    const float v = choice[e];
                    if (v == -INFINITY || to_key(v) < from)
                        continue;
                    const double c = exact_choice(r.softmax, r.max, r.sum,
                                                  load1<D>(a.logits, at + e),
                                                  a.bias ? a.bias[e] : 0.0f);
                    d2 = fmax(d2, fmin(d1, c));
                    d1 = fmax(d1, c);
                }
            }
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

template <class D, int V>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(RouteArgs a, int team)
{
    extern __shared__ float choice_sh[];       // [kWarps][E] with groups
    const uint32_t full = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= a.T)
        return;
    const uint64_t at = (uint64_t)t * a.E;

    // logits (-inf: out) and whether the bias moves the order at all
    float x[V];
    float blo = INFINITY, bhi = -INFINITY;
    bool bnan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < a.E ? load1<D>(a.logits, at + e) : -INFINITY;
        if (a.bias && e < a.E) {
            const float b = a.bias[e];
            if (b == -INFINITY)
                x[i] = -INFINITY;
            if (x[i] != -INFINITY) {
                blo = fminf(blo, b);
                bhi = fmaxf(bhi, b);
                bnan |= b != b;
            }
        }
    }
    bool by_logit = true;
    float bias0 = 0.0f;
    if (a.bias) {
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

    // ordering values: logits, or choice values
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        o[i] = x[i];
        if (!by_logit && x[i] != -INFINITY)
            o[i] = score_of(r, x[i]) + a.bias[lane + 32 * i];
    }
    uint32_t kept = full;
    float inv_size = 0.0f;
    if (a.G > 1) {
        float* choice = choice_sh + warp * a.E;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < a.E)
                choice[lane + 32 * i] = o[i];
        __syncwarp();
        kept = kept_groups<D>(a, r, choice, at, by_logit, bias0, base_err, lane, team);
        inv_size = 1.0f / (float)(a.E / a.G);
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = x[i] == -INFINITY ? 0u : to_key(o[i]);
        if (a.G > 1) {
            // e < 1024: (e + 1/2) / size in fp32 is below the next whole number
            const int g = (int)(((float)(lane + 32 * i) + 0.5f) * inv_size);
            if (g >= a.G || !(kept >> (g * team) & 1u))
                key[i] = 0u;
        }
    }

    int mine = -1;              // lane j: the j-th pick
    for (int j = 0; j < a.k; ++j) {
        uint32_t lb = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            lb = max(lb, key[i]);
        const uint32_t best = __reduce_max_sync(full, lb);
        if (best == 0)
            break;
        int pick = INT_MAX;
        bool exact = false;
        uint32_t thr = best;
        if (!by_logit && best > 1) {
            const float v = from_key(best);
            const float low = v - (base_err + 0x1p-22f * fabsf(v));
            thr = low > -INFINITY ? to_key(low) : best;
            int n = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                n += key[i] >= thr;
            const uint32_t who = __ballot_sync(full, n > 0);
            exact = __any_sync(full, n > 1) || (who & (who - 1)) != 0;
        }
        if (!exact) {
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                if (key[i] == best)
                    pick = lane + 32 * i;
            pick = (int)__reduce_min_sync(full, (uint32_t)pick);
        } else {
            if (r.softmax && r.sum == 0.0)
                r.sum = exact_sum<D>(a.logits, a.bias, at, a.E, r.max, lane);
            double c = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (key[i] >= thr) {
                    const int e = lane + 32 * i;
                    const double v = exact_choice(r.softmax, r.max, r.sum, x[i], a.bias[e]);
                    if (pick == INT_MAX || v > c) {
                        c = v;
                        pick = e;
                    }
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
        }
        if (lane == j)
            mine = pick;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == pick)
                key[i] = 0u;
    }

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
    int team = 32;              // lanes per group
    while (team * a.G > 32)
        team >>= 1;
    const unsigned grid = (unsigned)((a.T - 1) / kWarps + 1);
    const size_t smem = a.G > 1 ? sizeof(float) * kWarps * a.E : 0;
    const int per_lane = (a.E + 31) / 32;
    if (per_lane <= 1)
        route_kernel<D, 1><<<grid, 32 * kWarps, smem, s>>>(a, team);
    else if (per_lane <= 2)
        route_kernel<D, 2><<<grid, 32 * kWarps, smem, s>>>(a, team);
    else if (per_lane <= 4)
        route_kernel<D, 4><<<grid, 32 * kWarps, smem, s>>>(a, team);
    else if (per_lane <= 8)
        route_kernel<D, 8><<<grid, 32 * kWarps, smem, s>>>(a, team);
    else if (per_lane <= 16)
        route_kernel<D, 16><<<grid, 32 * kWarps, smem, s>>>(a, team);
    else
        route_kernel<D, 32><<<grid, 32 * kWarps, smem, s>>>(a, team);
    return cudaGetLastError();
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

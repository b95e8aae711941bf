// route_grouped.cuh -- MoE router with softmax or sigmoid scores, a selection
// bias, expert groups and scaled weights.  One warp per token.  Scores are
// doubles: a pick is decided between scores that lie next to each other, and
// fp32 scores would tie or swap where the definition does not.  They are
// compared as 64-bit integers of the same order, which costs no double
// operations.
#pragma once

#include "q8_device.cuh"
#include "route.cuh"

namespace q8 {

constexpr int kRouteMaxGroups = 32;
constexpr int kRouteGWarps = 4;

struct RouteArgs {
    const float *logits;  // [T][E]
    const float *bias;    // [E] or null
    int32_t *idx;         // [T][top_k]
    float *w;             // [T][top_k]
    int T, E, top_k, groups, keep, group_top;
    int sigmoid, renormalize;
    float scale;
};

// Order-preserving bits of a double, NaN as -inf, -0 as +0; above 0.
__device__ __forceinline__ unsigned long long ordered_key(double v) {
    v = isnan(v) ? -INFINITY : v + 0.0;
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ double key_double(unsigned long long k) {
    return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

__global__ void __launch_bounds__(32 * kRouteGWarps) route_grouped_kernel(const RouteArgs a) {
    __shared__ unsigned long long sel_s[kRouteGWarps][kRouteMaxE + 32];  // selection keys by group
    __shared__ double score_s[kRouteGWarps][kRouteMaxE];
    constexpr int PL = kRouteMaxE / 32;  // experts per lane
    pdl_wait_and_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRouteGWarps + warp;
    if (t >= a.T) return;
    const float *l = a.logits + (size_t)t * a.E;
    float v[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < a.E ? __ldg(l + e) : -INFINITY;
        if (isnan(v[i])) v[i] = -INFINITY;
    }
    double s[PL];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < PL; ++i) s[i] = lane + 32 * i < a.E ? 1.0 / (1.0 + exp(-(double)v[i])) : 0.0;
    } else {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            s[i] = v[i] == -INFINITY ? 0.0 : v[i] == mx ? 1.0 : exp((double)v[i] - (double)mx);
            z += s[i];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
#pragma unroll
        for (int i = 0; i < PL; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
    }
    // selection scores; key 0 marks an expert that cannot be picked (any more)
    const int size = a.E / a.groups;
    const int inv = (65536 + size - 1) / size;  // e / size = e * inv >> 16 for e * size < 2^16
    int lpg = 32;                               // lanes per group
    while (lpg * a.groups > 32) lpg >>= 1;
    unsigned long long key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < a.E ? ordered_key(s[i] + (a.bias ? (double)__ldg(a.bias + e) : 0.0)) : 0ull;
        if (e < a.E) {
            score_s[warp][e] = s[i];
            if (a.groups > 1) sel_s[warp][e + (e * inv >> 16) * lpg] = key[i];
        }
    }
    __syncwarp();
    if (a.groups > 1) {
        const int g = lane / lpg, sub = lane % lpg;
        unsigned long long b0 = 0, b1 = 0;  // the two largest
        if (g < a.groups)
            for (int e = sub; e < size; e += lpg) {
                const unsigned long long c = sel_s[warp][g * (size + lpg) + e];
                b1 = max(b1, min(b0, c));
                b0 = max(b0, c);
            }
        for (int off = lpg >> 1; off > 0; off >>= 1) {
            const unsigned long long o0 = __shfl_xor_sync(0xffffffffu, b0, off);
            const unsigned long long o1 = __shfl_xor_sync(0xffffffffu, b1, off);
            b1 = max(min(b0, o0), max(b1, o1));
            b0 = max(b0, o0);
        }
        const unsigned long long gk = a.group_top == 2 ? ordered_key(key_double(b0) + key_double(b1)) : b0;
        int better = 0;
        for (int o = 0; o < a.groups; ++o) {
            const unsigned long long ok = __shfl_sync(0xffffffffu, gk, o * lpg);
            better += ok > gk || (ok == gk && o < g);
        }
        const unsigned kept = __ballot_sync(0xffffffffu, g < a.groups && better < a.keep);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> ((e * inv >> 16) * lpg)) & 1u)) key[i] = 0ull;
        }
    }
    // top_k by key, ties to the lowest index
    int pick = 0;
    for (int k = 0; k < a.top_k; ++k) {
        unsigned long long bk = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < PL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
            }
        const unsigned hi = (unsigned)(bk >> 32), lo = (unsigned)bk;
        const unsigned mh = __reduce_max_sync(0xffffffffu, hi);
        const unsigned at = __ballot_sync(0xffffffffu, hi == mh);
        unsigned e;
        if ((at & (at - 1)) == 0) {  // nearly always: one lane has the largest high word
            e = __shfl_sync(0xffffffffu, (unsigned)(lane + 32 * bi), __ffs(at) - 1);
        } else {
            const unsigned ml = __reduce_max_sync(0xffffffffu, hi == mh ? lo : 0u);
            e = __reduce_min_sync(0xffffffffu, hi == mh && lo == ml ? (unsigned)(lane + 32 * bi) : ~0u);
        }
        if ((e & 31u) == (unsigned)lane) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if ((int)(e >> 5) == i) key[i] = 0ull;
        }
        if (lane == k) pick = (int)e;
    }
    double w = lane < a.top_k ? score_s[warp][pick] : 0.0;
    if (a.renormalize) {
        double sum = 0.0;
        for (int k = 0; k < a.top_k; ++k) sum += __shfl_sync(0xffffffffu, w, k);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < a.top_k) {
        a.idx[(size_t)t * a.top_k + lane] = pick;
        a.w[(size_t)t * a.top_k + lane] = (float)(w * (double)a.scale);
    }
}

}  // namespace q8

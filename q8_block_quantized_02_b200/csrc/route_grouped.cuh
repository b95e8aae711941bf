// route_grouped.cuh -- MoE router with softmax or sigmoid scores, a selection
// bias, expert groups and scaled weights.  One warp per token.  Scores are
// doubles: a pick is decided between scores that lie next to each other, and
// fp32 scores would tie or swap where the definition does not.  They are
// compared as 64-bit integers of the same order, which costs no double
// operations.
// Latency bounds it up to some hundred tokens (1 token of 60 experts 4.7 us, 16
// of 256 6.1 us, launches included), then the integer instructions: about 2000
// a token, 14.2 us for 4096 tokens of 256 experts in 8 groups (their bytes: 0.7
// us).
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

// Order-preserving bits of a double, NaN as -inf, -0 as +0.  Their high word
// is above 0 for every double.
__device__ __forceinline__ unsigned long long ordered_key(double v) {
    v = isnan(v) ? -INFINITY : v + 0.0;
    const int hi = __double2hiint(v), m = hi >> 31;
    return (unsigned long long)((unsigned)hi ^ ((unsigned)m | 0x80000000u)) << 32 | ((unsigned)__double2loint(v) ^ (unsigned)m);
}
__device__ __forceinline__ double key_double(unsigned long long k) {
    return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

// e^-x for x >= 0, 0 beyond 708 (whole warps): 2^(-(k + r) / 32) with k =
// round(32 log2(e) x), a table of 2^(-j / 32) held one entry per lane and the
// Taylor polynomial of 2^(-r / 32) to the sixth power (|r| <= 1/2: its
// remainder is below 2^-57).
__device__ __forceinline__ double exp_neg(double x, double tab) {
    constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52
    constexpr double a = 0.021660849392498290;     // ln 2 / 32
    const double y = fmin(x, 709.0) * 46.166241308446828;  // 32 log2(e)
    const double t = y + kMagic;
    const int k = __double2loint(t);
    const double r = y - (t - kMagic);
    double p = __fma_rn(r, a * a * a * a * a * a / 720, -a * a * a * a * a / 120);
    p = __fma_rn(r, p, a * a * a * a / 24);
    p = __fma_rn(r, p, -a * a * a / 6);
    p = __fma_rn(r, p, a * a / 2);
    p = __fma_rn(r, p, -a);
    p = __fma_rn(r, p, 1.0);
    const double w = p * __shfl_sync(0xffffffffu, tab, k & 31);
    return x > 708.0 ? 0.0 : __hiloint2double(__double2hiint(w) - ((k >> 5) << 20), __double2loint(w));
}

// 1 / d for 1 <= d: Newton's iteration from an fp32 estimate.
__device__ __forceinline__ double reciprocal(double d) {
    double y = (double)__fdividef(1.f, (float)d);
    y = __fma_rn(y, __fma_rn(-d, y, 1.0), y);
    return __fma_rn(y, __fma_rn(-d, y, 1.0), y);
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
    const double tab = exp2(-lane / 32.0);
    if (a.sigmoid) {
        // 1 / (1 + e^-l), below 0 as e^l / (1 + e^l)
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const double z = exp_neg(fabs((double)v[i]), tab);
            s[i] = (v[i] >= 0.f ? 1.0 : z) * reciprocal(1.0 + z);
        }
    } else {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const double w = exp_neg((double)mx - (double)v[i], tab);
            s[i] = v[i] == -INFINITY ? 0.0 : v[i] == mx ? 1.0 : w;
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
    // top_k by key, ties to the lowest index.  One key nearly always has the
    // largest high word alone, so a pick takes 32-bit maxima; the whole keys are
    // compared where it does not.
    int pick = 0;
    for (int k = 0; k < a.top_k; ++k) {
        unsigned mh = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) mh = max(mh, (unsigned)(key[i] >> 32));
        mh = __reduce_max_sync(0xffffffffu, mh);
        unsigned mine = 0;  // which of this lane's keys have it
#pragma unroll
        for (int i = 0; i < PL; ++i) mine |= (unsigned)(key[i] >> 32) == mh ? 1u << i : 0u;
        const unsigned at = __ballot_sync(0xffffffffu, mine != 0);
        const unsigned several = __ballot_sync(0xffffffffu, (mine & (mine - 1)) != 0);
        unsigned e;
        if ((at & (at - 1)) == 0 && several == 0) {
            e = __shfl_sync(0xffffffffu, (unsigned)lane + 32u * (unsigned)(__ffs(mine) - 1), __ffs(at) - 1);
        } else {
            unsigned lo = 0, bi = 0;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (((mine >> i) & 1u) && ((unsigned)key[i] > lo || !(mine & ((1u << i) - 1)))) {
                    lo = (unsigned)key[i];
                    bi = i;
                }
            const unsigned ml = __reduce_max_sync(0xffffffffu, mine ? lo : 0u);
            e = __reduce_min_sync(0xffffffffu, mine && lo == ml ? (unsigned)lane + 32u * bi : ~0u);
        }
        const unsigned hit = (e & 31u) == (unsigned)lane ? 1u << (e >> 5) : 0u;  // (a bit, so that key stays in registers)
#pragma unroll
        for (int i = 0; i < PL; ++i) key[i] = (hit >> i) & 1u ? 0ull : key[i];
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

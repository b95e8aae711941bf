// sample.cuh -- one token per row of logits: temperature, top-k, top-p, min-p,
// then the inverse CDF at a given uniform number.
//
// With m the row's largest logit and w_i = exp((l_i - m) / T), every filter
// keeps a prefix of the order (l descending, index ascending), so the kept set
// is "key > t, and the first `quota` of key == t" for one threshold key t
// (order-preserving bits of the fp32 logit).  The sums that decide -- the mass
// top-p cuts, the total and the running sum the uniform number meets -- are in
// fixed point: W_i = round(2^43 w_i) from a double exp, so a sum does not
// depend on its order and a pick is the same from run to run and for every
// split of the row.  (2^43: V <= 2^19 of them stay below 2^63; the rounding is
// 2^-44 of the largest weight, and a smaller weight is never drawn.)
//
// A row belongs to one thread-block cluster whose CTAs hold it in shared
// memory, so the logits are read once.  The threshold is found by rounds of a
// 2048-bin histogram (counts for top-k, mass for top-p) that the cluster adds
// up over distributed shared memory: two rounds of bins linear in the logit,
// then digits of the key while a bin still holds several values.
#pragma once

#include "q8q8_mma.cuh"
#include "q8_device.cuh"

namespace q8 {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBins = 2048;
constexpr int kSampleCoarse = kSampleBins / 32;
constexpr int kSampleMaxCluster = 16;
constexpr int kSampleMaxSlice = 32768;  // logits per CTA
constexpr double kSampleOne = 8796093022208.0;  // 2^43
constexpr double kSampleLive = 30.498476203173505;  // 44 ln 2: smaller weights are zero

typedef unsigned long long u64;

struct SampleArgs {
    const float *logits;       // [N][ld]
    const float *temperature;  // [N] or null (1)
    const int32_t *top_k;      // [N] or null (off)
    const float *top_p;        // [N] or null (off)
    const float *min_p;        // [N] or null (off)
    const float *u;            // [N]
    int32_t *token;            // [N]
    float *prob;               // [N] or null
    int64_t ld;
    int V, slice;              // logits per CTA
};

struct SampleShared {
    u64 mass[2][kSampleBins];
    uint32_t cnt[2][kSampleBins];
    u64 cmass[2][kSampleCoarse];
    uint32_t ccnt[2][kSampleCoarse];
    u64 best;      // this CTA's largest logit and its index (read by the cluster)
    u64 fin_mass;  // this CTA's mass above the threshold, and its count of equals
    uint32_t fin_eq;
    u64 wmass[kSampleWarps];
    uint32_t weq[kSampleWarps];
    // results of a step for the whole CTA
    u64 gbest, total, before, target, z;
    uint32_t count, bin, lo, hi, quota;
    int found;
};

__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
__device__ __forceinline__ T warp_incl_scan(T v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Fixed-point weight of a logit (mx: the row's largest).
struct SampleWeight {
    float mx;
    double inv_t;
    __device__ __forceinline__ double real(float l) const {
        return l == mx ? 1.0 : exp(((double)l - (double)mx) * inv_t);
    }
    __device__ __forceinline__ u64 fixed(float l) const { return __double2ull_rn(real(l) * kSampleOne); }
};

// A round's bins: bin 0 holds the largest logits, and the bin never falls as
// the logit falls (every step of the linear form is a monotone fp32 operation;
// the conversion clamps, and takes the NaN of inf - inf or 0 * inf to bin 0).
struct SampleBinning {
    float mx, scale, v0, mult;
    uint32_t hi;
    int shift;  // < 0: linear
    __device__ __forceinline__ uint32_t operator()(uint32_t key) const {
        if (shift >= 0) return (hi - key) >> shift;
        const float v = __fmul_rn(__fsub_rn(__fmul_rn(__fsub_rn(mx, key_logit(key)), scale), v0), mult);
        return (uint32_t)min(max(__float2int_rz(v), 0), kSampleBins - 1);
    }
};

// The least key in [lo, hi] whose bin is <= b (one whole warp; bins fall as
// keys rise, and bin(hi) <= b).
__device__ __forceinline__ uint32_t least_key_of_bin(const SampleBinning &bin, uint32_t lo, uint32_t hi, uint32_t b,
                                                     int lane) {
    while (lo < hi) {  // 32 probes a step
        const u64 span = (u64)hi - lo;
        const uint32_t k = lo + (uint32_t)(span * lane / 32);  // k < hi
        const unsigned in = __ballot_sync(0xffffffffu, bin(k) <= b);
        if (in & 1u) return lo;
        const int f = in ? __ffs(in) - 1 : 32;  // first probe inside
        const uint32_t nlo = lo + (uint32_t)(span * (f - 1) / 32) + 1;
        const uint32_t nhi = f == 32 ? hi : lo + (uint32_t)(span * f / 32);
        lo = nlo;
        hi = nhi;
    }
    return lo;
}

// One CTA's state while it looks for thresholds.
struct SampleRow {
    SampleShared *sh;
    const float *l;  // this CTA's logits in shared memory
    int n;           // how many
    uint32_t CL;
    int tid, warp, lane;
    int round;       // histogram buffer to use next
    SampleWeight weight;
    float scale;     // bins per unit of logit, first round
};

// Narrows [lo, hi] to the threshold key of a count (MASS false: the first
// `target` elements) or of a mass (MASS true; top_p of the interval's whole
// mass less `excess`).  Returns the threshold in *lo_out and how many equals
// are kept in *quota (0xffffffff: all); false when the whole interval stays.
template <bool MASS>
__device__ bool sample_select(SampleRow &s, uint32_t lo, uint32_t hi, u64 target, double top_p, u64 excess,
                              uint32_t *lo_out, uint32_t *quota, u64 *total_mass) {
    SampleShared &sh = *s.sh;
    u64 before = 0;  // of the elements above the interval
    SampleBinning bin{s.weight.mx, s.scale, 0.f, 1.f, hi, -1};
    for (int it = 0;; ++it) {
        const int buf = s.round & 1;
        ++s.round;
        for (int i = s.tid; i < kSampleBins; i += kSampleThreads) {
            sh.cnt[buf][i] = 0;
            if (MASS) sh.mass[buf][i] = 0;
        }
        __syncthreads();
        for (int i = s.tid; i < s.n; i += kSampleThreads) {
            const float l = s.l[i];
            const uint32_t k = logit_key(l);
            if (k >= lo && k <= hi) {
                const uint32_t b = bin(k);
                atomicAdd(&sh.cnt[buf][b], 1u);
                if (MASS) atomicAdd(&sh.mass[buf][b], s.weight.fixed(l));
            }
        }
        __syncthreads();
        for (int g = s.warp; g < kSampleCoarse; g += kSampleWarps) {
            const uint32_t c = warp_sum(sh.cnt[buf][g * 32 + s.lane]);
            const u64 m = MASS ? warp_sum(sh.mass[buf][g * 32 + s.lane]) : 0;
            if (s.lane == 0) {
                sh.ccnt[buf][g] = c;
                sh.cmass[buf][g] = m;
            }
        }
        cluster_sync_all();
        if (s.warp < 2) {
            // both warps find the bin; warp 0 then looks for the bin's least
            // key, warp 1 for its largest
            u64 c0 = 0, c1 = 0;  // coarse groups 2 lane, 2 lane + 1
            for (uint32_t p = 0; p < s.CL; ++p) {
                if (MASS) {
                    const uint32_t a = map_to_rank(smem_u32(&sh.cmass[buf][2 * s.lane]), p);
                    c0 += ld_cluster_u64(a);
                    c1 += ld_cluster_u64(a + 8);
                } else {
                    const uint32_t a = map_to_rank(smem_u32(&sh.ccnt[buf][2 * s.lane]), p);
                    c0 += ld_cluster_u32(a);
                    c1 += ld_cluster_u32(a + 4);
                }
            }
            const u64 inc = warp_incl_scan(c0 + c1, s.lane);
            const u64 all = __shfl_sync(0xffffffffu, inc, 31);
            if (MASS && it == 0) {
                const double z = (double)(all - excess);
                target = (u64)ceil(top_p * z);
                if (target < 1) target = 1;
            }
            u64 b4 = before;
            uint32_t fine = 0, c = 0;
            const bool cross = before + all >= target && all > 0;
            if (cross) {
                const u64 ex = before + inc - c0 - c1;
                const bool in0 = ex < target && target <= ex + c0;
                const bool in1 = ex + c0 < target && target <= ex + c0 + c1;
                const int src = __ffs(__ballot_sync(0xffffffffu, in0 || in1)) - 1;
                const uint32_t g = __shfl_sync(0xffffffffu, 2 * s.lane + (in1 ? 1 : 0), src);
                b4 = __shfl_sync(0xffffffffu, in1 ? ex + c0 : ex, src);
                u64 fm = 0;
                uint32_t fc = 0;
                for (uint32_t p = 0; p < s.CL; ++p) {
                    fc += ld_cluster_u32(map_to_rank(smem_u32(&sh.cnt[buf][g * 32 + s.lane]), p));
                    if (MASS) fm += ld_cluster_u64(map_to_rank(smem_u32(&sh.mass[buf][g * 32 + s.lane]), p));
                }
                const u64 val = MASS ? fm : fc;
                const u64 fi = b4 + warp_incl_scan(val, s.lane);
                const int f = __ffs(__ballot_sync(0xffffffffu, fi - val < target && target <= fi)) - 1;
                fine = g * 32 + f;
                c = __shfl_sync(0xffffffffu, fc, f);
                b4 = __shfl_sync(0xffffffffu, fi - val, f);
                // the bin's keys
                uint32_t k;
                if (s.warp == 0)
                    k = bin.shift < 0 ? least_key_of_bin(bin, lo, hi, fine, s.lane)
                                      : (uint32_t)max((long long)lo, (long long)hi - (((long long)fine + 1) << bin.shift) + 1);
                else if (bin.shift >= 0)
                    k = hi - (fine << bin.shift);
                else
                    k = bin(hi) == fine ? hi : least_key_of_bin(bin, lo, hi, fine - 1, s.lane) - 1;
                if (s.lane == 0) (s.warp == 0 ? sh.lo : sh.hi) = k;
            }
            if (s.warp == 0 && s.lane == 0) {
                sh.found = cross;
                sh.before = b4;
                sh.count = c;
                sh.bin = fine;
                sh.target = target;
                sh.total = all;
            }
        }
        __syncthreads();
        const bool cross = sh.found != 0;
        const uint32_t nlo = sh.lo, nhi = sh.hi, c = sh.count, fine = sh.bin;
        before = sh.before;
        target = sh.target;
        if (it == 0) *total_mass = sh.total;
        __syncthreads();
        if (!cross) return false;
        *lo_out = nlo;
        if (MASS ? c == 1 : target - before == c) {
            *quota = 0xffffffffu;
            return true;
        }
        if (nlo == nhi) {
            if (MASS) {
                const u64 w = s.weight.fixed(key_logit(nlo));
                *quota = (uint32_t)((target - before + w - 1) / w);
            } else {
                *quota = (uint32_t)(target - before);
            }
            return true;
        }
        lo = nlo;
        hi = nhi;
        if (it == 0 && fine < kSampleBins - 1) {  // (the last bin takes all that lies beyond)
            bin.v0 = (float)fine;
            bin.mult = (float)kSampleBins;
        } else {
            const int bits = 32 - __clz(hi - lo);
            bin.shift = max(0, bits - 11);
            bin.hi = hi;
        }
    }
}

__global__ void __launch_bounds__(kSampleThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t sample_smem[];
    SampleShared &sh = *reinterpret_cast<SampleShared *>(sample_smem);
    float *buf = reinterpret_cast<float *>(sample_smem + sizeof(SampleShared));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t CL;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(CL));
    const uint32_t rank = cluster_ctarank();
    const int row = blockIdx.x / CL;
    pdl_wait_and_trigger();

    // this CTA's logits: NaN counts as -inf, -0 as +0; the largest, lowest index first
    const int i0 = min(a.V, (int)rank * a.slice);
    const int n = min(a.V, i0 + a.slice) - i0;
    const float *src = a.logits + (int64_t)row * a.ld + i0;
    u64 best = 0;
    for (int i = tid; i < n; i += kSampleThreads) {
        float v = __ldg(src + i) + 0.f;
        if (isnan(v)) v = -INFINITY;
        buf[i] = v;
        const u64 k = ((u64)logit_key(v) << 32) | (0xffffffffu - (uint32_t)(i0 + i));
        best = k > best ? k : best;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
        best = o > best ? o : best;
    }
    if (lane == 0) sh.wmass[warp] = best;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kSampleWarps; ++w) best = sh.wmass[w] > best ? sh.wmass[w] : best;
        sh.best = best;
    }
    cluster_sync_all();
    if (warp == 0) {
        best = lane < (int)CL ? ld_cluster_u64(map_to_rank(smem_u32(&sh.best), lane)) : 0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        if (lane == 0) sh.gbest = best;
    }
    __syncthreads();
    best = sh.gbest;
    const uint32_t key_max = (uint32_t)(best >> 32);
    const float mx = key_logit(key_max);
    float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
    if (mx == -INFINITY || !(temp > 0.f)) {  // nothing to draw from, or greedy
        if (rank == 0 && tid == 0) {
            a.token[row] = mx == -INFINITY ? -1 : (int32_t)(0xffffffffu - (uint32_t)best);
            if (a.prob) a.prob[row] = mx == -INFINITY ? 0.f : 1.f;
        }
        cluster_sync_all();  // sh.best is read by the whole cluster
        return;
    }
    temp = fminf(temp, 3.402823466e38f);

    SampleRow s;
    s.sh = &sh;
    s.l = buf;
    s.n = n;
    s.CL = CL;
    s.tid = tid;
    s.warp = warp;
    s.lane = lane;
    s.round = 0;
    s.weight = SampleWeight{mx, 1.0 / (double)temp};
    s.scale = (float)(kSampleBins / (kSampleLive * (double)temp));

    // threshold: the weight's cut-off, then each filter raises it
    const uint32_t key_low = logit_key(-3.402823466e38f);
    uint32_t t = logit_key(__double2float_ru((double)mx - kSampleLive * (double)temp) + 0.f);
    t = max(t, key_low);
    uint32_t quota = 0xffffffffu;
    u64 excess = 0, unused;
    const int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
    if (top_k > 0 && top_k < a.V) {
        uint32_t nt, nq;
        if (sample_select<false>(s, t, key_max, (u64)top_k, 0.0, 0, &nt, &nq, &unused)) {
            t = nt;
            quota = nq;
            if (quota != 0xffffffffu) {  // equals of the threshold beyond the quota
                const uint32_t eq = sh.count;
                excess = (u64)(eq - quota) * s.weight.fixed(key_logit(t));
            }
        }
    }
    const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
    if (top_p < 1.f) {
        uint32_t nt, nq;
        if (sample_select<true>(s, t, key_max, 0, (double)top_p, excess, &nt, &nq, &unused)) {
            t = nt;
            quota = nq;
        }
    }
    const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
    if (min_p > 0.f) {
        const double c = (double)mx + (double)temp * log((double)fminf(min_p, 1.f));
        const uint32_t k = min(key_max, logit_key(__double2float_ru(c) + 0.f));
        if (k > t) {
            t = k;
            quota = 0xffffffffu;
        }
    }

    // kept mass: a warp takes a contiguous part of the slice
    const int seg = ((a.slice + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
    const int s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
    const u64 wt = quota == 0xffffffffu ? 0 : s.weight.fixed(key_logit(t));
    {
        u64 m = 0;
        uint32_t eq = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint32_t k = logit_key(buf[i]);
            if (k > t || (k == t && quota == 0xffffffffu)) m += s.weight.fixed(buf[i]);
            if (k == t) ++eq;
        }
        m = warp_sum(m);
        eq = quota == 0xffffffffu ? 0 : warp_sum(eq);
        if (lane == 0) {
            sh.wmass[warp] = m;
            sh.weq[warp] = eq;
        }
    }
    __syncthreads();
    if (tid == 0) {
        u64 m = 0;
        uint32_t eq = 0;
        for (int w = 0; w < kSampleWarps; ++w) {
            m += sh.wmass[w];
            eq += sh.weq[w];
        }
        sh.fin_mass = m;
        sh.fin_eq = eq;
    }
    cluster_sync_all();
    // which CTA, then which warp's part, the uniform number falls into
    if (warp == 0) {
        u64 m = 0;
        uint32_t eq = 0;
        if (lane < (int)CL) {
            m = ld_cluster_u64(map_to_rank(smem_u32(&sh.fin_mass), lane));
            eq = ld_cluster_u32(map_to_rank(smem_u32(&sh.fin_eq), lane));
        }
        uint32_t pre = warp_incl_scan(eq, lane) - eq;
        uint32_t left = quota > pre ? quota - pre : 0;  // equals this CTA may still keep
        u64 km = m + (u64)min(left, eq) * wt;
        u64 inc = warp_incl_scan(km, lane);
        const u64 z = __shfl_sync(0xffffffffu, inc, 31);
        float u = __ldg(a.u + row);
        u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
        u64 r = (u64)((double)u * (double)z);
        if (r > z - 1) r = z - 1;
        const int c = __ffs(__ballot_sync(0xffffffffu, inc - km <= r && r < inc)) - 1;
        r -= __shfl_sync(0xffffffffu, inc - km, c);
        left = __shfl_sync(0xffffffffu, left, c);
        int w = -1;
        if (c == (int)rank) {
            m = lane < kSampleWarps ? sh.wmass[lane] : 0;
            eq = lane < kSampleWarps ? sh.weq[lane] : 0;
            pre = warp_incl_scan(eq, lane) - eq;
            const uint32_t wl = left > pre ? left - pre : 0;
            km = m + (u64)min(wl, eq) * wt;
            inc = warp_incl_scan(km, lane);
            w = __ffs(__ballot_sync(0xffffffffu, inc - km <= r && r < inc)) - 1;
            r -= __shfl_sync(0xffffffffu, inc - km, w);
            left = __shfl_sync(0xffffffffu, wl, w);
        }
        if (lane == 0) {
            sh.found = w;
            sh.target = r;
            sh.quota = left;
            sh.z = z;
        }
    }
    __syncthreads();
    const int part = sh.found;
    if (part >= 0) {  // this CTA holds the token: every thread takes a few elements of the part
        const u64 r = sh.target, z = sh.z;
        const uint32_t left = sh.quota;
        const int per = (seg + kSampleThreads - 1) / kSampleThreads;
        const int e0 = min(n, part * seg) + tid * per;
        const int e1 = min(min(n, (part + 1) * seg), e0 + per);
        u64 m = 0;
        uint32_t eq = 0;
        for (int i = e0; i < e1; ++i) {
            const uint32_t k = logit_key(buf[i]);
            if (k > t || (k == t && quota == 0xffffffffu)) m += s.weight.fixed(buf[i]);
            if (k == t && quota != 0xffffffffu) ++eq;
        }
        // sums of the threads before this one, equals first
        uint32_t pe = warp_incl_scan(eq, lane);
        __syncthreads();
        if (lane == 31) sh.weq[warp] = pe;
        __syncthreads();
        pe -= eq;
        for (int w = 0; w < warp; ++w) pe += sh.weq[w];
        const uint32_t tl = left > pe ? left - pe : 0;
        const u64 km = m + (u64)min(tl, eq) * wt;
        u64 inc = warp_incl_scan(km, lane);
        if (lane == 31) sh.wmass[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) inc += sh.wmass[w];
        if (inc - km <= r && r < inc) {
            u64 run = inc - km;
            uint32_t q = tl;
            for (int i = e0; i < e1; ++i) {
                const uint32_t k = logit_key(buf[i]);
                u64 w = 0;
                if (k > t || (k == t && quota == 0xffffffffu))
                    w = s.weight.fixed(buf[i]);
                else if (k == t && q > 0) {
                    w = wt;
                    --q;
                }
                if (run <= r && r < run + w) {
                    a.token[row] = i0 + i;
                    if (a.prob) a.prob[row] = (float)(s.weight.real(buf[i]) * kSampleOne / (double)z);
                }
                run += w;
            }
        }
    }
    cluster_sync_all();  // this CTA's shared memory is read by the whole cluster
}

}  // namespace q8

// sample.cuh -- one token per row of logits: temperature, top-k, top-p, min-p,
// then the inverse CDF at a given uniform number.
//
// With m the row's largest logit and w_i = exp((l_i - m) / T), every filter
// keeps a prefix of the order (l descending, index ascending): the kept set is
// K >= Kt for one threshold of the composite order key K_i = (order-preserving
// bits of l_i) << 32 | ~i.  The sums that decide -- the mass top-p cuts, the
// total and the running sum the uniform number meets -- are in fixed point:
// W_i = round(2^43 w_i), w_i in double, so a sum does not depend on its order
// and a pick is the same from run to run and for every split of the row.
// (2^43: V <= 2^19 of them stay below 2^63; the rounding is 2^-44 of the
// largest weight, and a smaller weight is never drawn.)
//
// A row belongs to one thread-block cluster whose CTAs hold it in shared
// memory, so the logits are read once.  A filter's threshold comes from a
// 2048-bin histogram of the row (counts for top-k, mass for top-p) that the
// cluster adds up over distributed shared memory; the crossing bin's elements
// -- or everything down to that bin, when that is a short list -- are then
// copied to every CTA, which settles the threshold among them on its own.  So a
// row takes two or three cluster barriers; only runs of ties longer than the
// list take more rounds.
#pragma once

#include "q8q8_mma.cuh"
#include "q8_device.cuh"

namespace q8 {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBins = 2048;
constexpr int kSampleGroup = 64;  // bins per group
constexpr int kSampleGroups = kSampleBins / kSampleGroup;
constexpr int kSampleList = 1024;
constexpr int kSampleMaxCluster = 16;
constexpr int kSampleMaxSlice = 32768;  // logits per CTA
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
    int V, slice;              // slice: logits per CTA
};

// What the other CTAs of the cluster write here.
struct SampleInbox {
    u64 gmass[kSampleGroups];
    uint32_t gcnt[kSampleGroups];
    u64 best;  // largest composite key
    u64 kept;  // kept mass, or the mass above the crossing bin
};

struct SampleShared {
    u64 mass[kSampleBins];     // read by the cluster
    uint32_t cnt[kSampleBins];
    u64 list[kSampleList];     // written by the cluster
    uint32_t list_n[2];        // entries given out (rank 0's counts for all), per filter
    u64 wsum[kSampleWarps];
    u64 gm[32];                // group sums of a list's histogram
    u64 tiny[32];
    uint32_t tiny_n;
    // results of one thread or warp for the whole CTA
    u64 before, lo, hi, target, val;
    u64 tot[kSampleMaxCluster];
    uint32_t count, above;
    int bin;
};

__host__ __device__ inline size_t sample_smem_bytes(int slice, int cl) {
    return sizeof(SampleShared) + (size_t)cl * sizeof(SampleInbox) + (size_t)slice * 4;
}

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
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t atom_cluster_add(uint32_t addr, uint32_t v) {
    uint32_t o;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(addr), "r"(v) : "memory");
    return o;
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

// Fixed-point weight of a logit (mx: the row's largest).  2^(-(k + r) / 32)
// with k = round(32 log2(e) (mx - l) / T): a table of 2^(-j / 32) held one
// entry per lane, and the Taylor polynomial of 2^(-r / 32) to the fifth power
// (|r| <= 1/2: its remainder is below 2^-48), so 12 double operations.
// Whole warps only; a weight below the live threshold comes out as garbage.
struct SampleWeight {
    float mx;
    double c;    // 32 log2(e) / T
    double tab;  // 2^(-lane / 32)
    __device__ __forceinline__ u64 operator()(float l) const {
        constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52
        constexpr double a = 0.021660849392498290;     // ln 2 / 32
        const double d = (double)mx - (double)l;
        const double t = __fma_rn(d, c, kMagic);
        const int k = __double2loint(t);
        const double r = __fma_rn(d, c, -(t - kMagic));
        double p = __fma_rn(r, -a * a * a * a * a / 120, a * a * a * a / 24);
        p = __fma_rn(r, p, -a * a * a / 6);
        p = __fma_rn(r, p, a * a / 2);
        p = __fma_rn(r, p, -a);
        p = __fma_rn(r, p, 1.0);
        const double w = p * __shfl_sync(0xffffffffu, tab, k & 31);
        const double s = __hiloint2double(__double2hiint(w) + ((43 - (k >> 5)) << 20), __double2loint(w));
        const u64 f = (u64)__double_as_longlong(s + 4503599627370496.0) & 0xfffffffffffffull;  // + 2^52
        return l == mx ? 1ull << 43 : f;
    }
};

// The histogram's bins: 128 to a unit of (mx - l) / T down to 14, then 16 to a
// unit, and the last bin takes what lies beyond.  Bin 0 holds the largest
// logits and the bin never falls as the logit falls: every step is a monotone
// fp32 operation, the conversion clamps, and it takes the NaN of inf - inf or
// 0 * inf to bin 0.  (14 units below the top a token of 2^19 holds under one
// part in 2^20 of the mass; finer bins above make the crossing bin's list
// short.)
struct SampleBinning {
    float mx, scale;  // 128 / T
    __device__ __forceinline__ int operator()(float l) const {
        const float v = __fmul_rn(__fsub_rn(mx, l), scale);
        const float s = v < 1792.f ? v : __fadd_rn(1792.f, __fmul_rn(__fsub_rn(v, 1792.f), 0.125f));
        return min(max(__float2int_rz(s), 0), kSampleBins - 1);
    }
};

// The least key in [lo, hi] whose bin is <= b; hi + 1 when there is none.
// A whole warp, 32 probes a step.
__device__ __forceinline__ u64 least_key_of_bin(const SampleBinning &bin, uint32_t lo, uint32_t hi, int b, int lane) {
    if (bin(key_logit(hi)) > b) return (u64)hi + 1;
    while (lo < hi) {
        const u64 span = (u64)hi - lo;
        const unsigned in = __ballot_sync(0xffffffffu, bin(key_logit(lo + (uint32_t)(span * lane / 32))) <= b);
        if (in & 1u) return lo;
        const int f = in ? __ffs(in) - 1 : 32;  // first probe inside
        if (f < 32) hi = lo + (uint32_t)(span * f / 32);
        lo += (uint32_t)(span * (f - 1) / 32) + 1;
    }
    return lo;
}

struct SampleRow {
    SampleShared *sh;
    SampleInbox *inbox;  // [CL]
    const float *l;      // this CTA's logits
    int n, i0;           // how many, and the first one's index
    uint32_t CL, rank;
    int tid, warp, lane;
    SampleWeight weight;
    SampleBinning bin;
    __device__ __forceinline__ u64 composite(int i) const {
        return ((u64)logit_key(l[i]) << 32) | (0xffffffffu - (uint32_t)(i0 + i));
    }
};

// Among the list's entries e >= kt, in descending order of e (by_index: in
// ascending index order), the one where the running count (MASS: mass), from
// `before`, reaches `target`: the only entries that can are those of order
// keys [lo, hi], and one of them does.  Returns its order key (e, or its low
// half).  Whole CTA.
template <bool MASS>
__device__ u64 sample_list_select(const SampleRow &s, int n, u64 kt, bool by_index, u64 lo, u64 hi, u64 before,
                                  u64 target) {
    SampleShared &sh = *s.sh;
    uint32_t count = (uint32_t)n;
    while (count > 32) {
        const int bits = 64 - __clzll((long long)(hi - lo));
        const int shift = max(0, bits - 10);  // 1024 bins, 32 groups of 32
        for (int i = s.tid; i < 1024; i += kSampleThreads) {
            sh.cnt[i] = 0;
            if (MASS) sh.mass[i] = 0;
        }
        __syncthreads();
        for (int i = s.tid; i - s.lane < n; i += kSampleThreads) {
            const u64 e = i < n ? sh.list[i] : 0;
            const u64 o = by_index ? (uint32_t)e : e;
            const u64 w = MASS ? s.weight(key_logit((uint32_t)(e >> 32))) : 0;
            if (i < n && e >= kt && o >= lo && o <= hi) {
                const int b = (int)((hi - o) >> shift);
                atomicAdd(&sh.cnt[b], 1u);
                if (MASS) atomicAdd(&sh.mass[b], w);
            }
        }
        __syncthreads();
        for (int g = s.warp; g < 32; g += kSampleWarps) {
            const u64 v = warp_sum(MASS ? sh.mass[g * 32 + s.lane] : (u64)sh.cnt[g * 32 + s.lane]);
            if (s.lane == 0) sh.gm[g] = v;
        }
        __syncthreads();
        if (s.warp == 0) {
            u64 v = sh.gm[s.lane];
            u64 inc = before + warp_incl_scan(v, s.lane);
            const int g = __ffs(__ballot_sync(0xffffffffu, inc - v < target && target <= inc)) - 1;
            const u64 b4 = __shfl_sync(0xffffffffu, inc - v, g);
            const uint32_t c = sh.cnt[g * 32 + s.lane];
            v = MASS ? sh.mass[g * 32 + s.lane] : c;
            inc = b4 + warp_incl_scan(v, s.lane);
            if (inc - v < target && target <= inc) {
                const u64 top = hi - ((u64)(g * 32 + s.lane) << shift);
                const u64 span = (1ull << shift) - 1;
                sh.hi = top;
                sh.lo = top - lo > span ? top - span : lo;
                sh.before = inc - v;
                sh.count = c;
            }
        }
        __syncthreads();
        lo = sh.lo;
        hi = sh.hi;
        before = sh.before;
        count = sh.count;
        __syncthreads();
    }
    if (s.tid == 0) sh.tiny_n = 0;
    __syncthreads();
    for (int i = s.tid; i < n; i += kSampleThreads) {
        const u64 e = sh.list[i];
        const u64 o = by_index ? (uint32_t)e : e;
        if (e >= kt && o >= lo && o <= hi) sh.tiny[atomicAdd(&sh.tiny_n, 1u) & 31u] = e;
    }
    __syncthreads();
    if (s.warp == 0) {
        const int tn = min((int)sh.tiny_n, 32);
        const u64 e = s.lane < tn ? sh.tiny[s.lane] : 0;
        const u64 o = by_index ? (uint32_t)e : e;
        u64 w = MASS ? s.weight(key_logit((uint32_t)(e >> 32))) : 1;
        if (s.lane >= tn) w = 0;
        u64 ex = before;
        for (int j = 0; j < tn; ++j) {
            const u64 oj = __shfl_sync(0xffffffffu, o, j), wj = __shfl_sync(0xffffffffu, w, j);
            if (oj > o) ex += wj;
        }
        if (s.lane < tn && ex < target && target <= ex + w) sh.val = o;
    }
    __syncthreads();
    const u64 r = sh.val;
    __syncthreads();
    return r;
}

// The mass of the list's entries e >= kt.  Whole CTA.
__device__ u64 sample_list_mass(const SampleRow &s, int n, u64 kt) {
    SampleShared &sh = *s.sh;
    u64 m = 0;
    for (int i = s.tid; i - s.lane < n; i += kSampleThreads) {
        const u64 e = i < n ? sh.list[i] : 0;
        const u64 w = s.weight(key_logit((uint32_t)(e >> 32)));
        if (i < n && e >= kt) m += w;
    }
    m = warp_sum(m);
    if (s.lane == 0) sh.wsum[s.warp] = m;
    __syncthreads();
    m = 0;
    for (int w = 0; w < kSampleWarps; ++w) m += sh.wsum[w];
    __syncthreads();
    return m;
}

enum { kSampleWhole, kSampleShort, kSampleFound };

// One filter: the threshold composite key in [lo, hi] of a count (the first
// `target`) or, MASS, of a mass (top_p of the interval's).  Returns
//   kSampleFound: *kt set, the same in every CTA (in_first: settled in the
//     first histogram, whose per-CTA mass above the crossing bin is in
//     inbox[].kept and whose list of n entries is still there);
//   kSampleShort: the list holds every element that may be kept (n of them, in
//     rank 0 only), [*blo, *bhi] the crossing bin's keys, *before and *target
//     its sums; *bhi < *blo when the filter cuts nothing;
//   kSampleWhole: the filter cuts nothing and the elements are many.
template <bool MASS>
__device__ int sample_filter(const SampleRow &s, u64 lo, u64 hi, u64 target, double top_p, int slot, u64 *kt, int *n_list,
                             u64 *blo, u64 *bhi, u64 *before_out, u64 *target_out, bool *in_first) {
    SampleShared &sh = *s.sh;
    u64 before = 0;
    for (int it = 0;; ++it) {
        const int bits = 64 - __clzll((long long)(hi - lo));
        const int shift = max(0, bits - 11);  // later rounds: digits of the composite key
        if (it > 0) cluster_sync_all();       // the histogram is no longer read
        for (int i = s.tid; i < kSampleBins; i += kSampleThreads) {
            sh.cnt[i] = 0;
            if (MASS) sh.mass[i] = 0;
        }
        __syncthreads();
#pragma unroll 4
        for (int i = s.tid; i - s.lane < s.n; i += kSampleThreads) {
            const float l = i < s.n ? s.l[i] : 0.f;
            const u64 k = ((u64)logit_key(l) << 32) | (0xffffffffu - (uint32_t)(s.i0 + i));
            const u64 w = MASS ? s.weight(l) : 0;
            if (i < s.n && k >= lo && k <= hi) {
                const int b = it == 0 ? s.bin(l) : (int)((hi - k) >> shift);
                atomicAdd(&sh.cnt[b], 1u);
                if (MASS) atomicAdd(&sh.mass[b], w);
            }
        }
        __syncthreads();
        for (int g = s.warp; g < kSampleGroups; g += kSampleWarps) {
            const int b = g * kSampleGroup + s.lane;
            const uint32_t c = warp_sum(sh.cnt[b] + sh.cnt[b + 32]);
            const u64 m = MASS ? warp_sum(sh.mass[b] + sh.mass[b + 32]) : 0;
            if (s.lane < (int)s.CL) {
                st_cluster_u32(map_to_rank(smem_u32(&s.inbox[s.rank].gcnt[g]), s.lane), c);
                if (MASS) st_cluster_u64(map_to_rank(smem_u32(&s.inbox[s.rank].gmass[g]), s.lane), m);
            }
        }
        cluster_sync_all();
        // the crossing group, then its bins from all CTAs (two warps, a bin a lane and warp)
        if (s.warp < 2) {
            u64 v = 0;
            uint32_t c = 0;
            for (uint32_t p = 0; p < s.CL; ++p) {
                c += s.inbox[p].gcnt[s.lane];
                if (MASS) v += s.inbox[p].gmass[s.lane];
            }
            if (!MASS) v = c;
            const u64 inc = warp_incl_scan(v, s.lane);
            const uint32_t cinc = warp_incl_scan(c, s.lane);
            const u64 all = __shfl_sync(0xffffffffu, inc, 31);
            const uint32_t call = __shfl_sync(0xffffffffu, cinc, 31);
            if (MASS && it == 0) {
                target = (u64)ceil(top_p * (double)all);
                if (target < 1) target = 1;
            }
            int b = -1;
            uint32_t bc = 0, ba = call;
            u64 b4 = before + all;
            if (target <= before + all) {
                const unsigned cross = __ballot_sync(0xffffffffu, before + inc - v < target && target <= before + inc);
                const int g = __ffs(cross) - 1;
                b4 = before + __shfl_sync(0xffffffffu, inc - v, g);
                ba = __shfl_sync(0xffffffffu, cinc - c, g);
                uint32_t fc[2] = {0, 0};
                u64 fm[2] = {0, 0};
#pragma unroll
                for (uint32_t p = 0; p < kSampleMaxCluster; ++p) {
                    if (p < s.CL) {
                        const uint32_t ac = map_to_rank(smem_u32(&sh.cnt[g * kSampleGroup + s.lane]), p);
                        fc[0] += ld_cluster_u32(ac);
                        fc[1] += ld_cluster_u32(ac + 128);
                        if (MASS) {
                            const uint32_t am = map_to_rank(smem_u32(&sh.mass[g * kSampleGroup + s.lane]), p);
                            fm[0] += ld_cluster_u64(am);
                            fm[1] += ld_cluster_u64(am + 256);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u64 x = MASS ? fm[h] : fc[h];
                    const u64 xi = b4 + warp_incl_scan(x, s.lane);
                    const uint32_t ci = ba + warp_incl_scan(fc[h], s.lane);
                    const unsigned at = __ballot_sync(0xffffffffu, xi - x < target && target <= xi);
                    if (b < 0 && at) {
                        const int f = __ffs(at) - 1;
                        b = g * kSampleGroup + 32 * h + f;
                        bc = __shfl_sync(0xffffffffu, fc[h], f);
                        b4 = __shfl_sync(0xffffffffu, xi - x, f);
                        ba = __shfl_sync(0xffffffffu, ci - fc[h], f);
                    } else if (b < 0) {
                        b4 = __shfl_sync(0xffffffffu, xi, 31);
                        ba = __shfl_sync(0xffffffffu, ci, 31);
                    }
                }
                // the bin's keys: warp 0 the least, warp 1 the largest
                u64 k;
                if (it > 0)
                    k = s.warp == 0 ? (hi - lo >> shift > (u64)b ? hi - (((u64)b + 1) << shift) + 1 : lo)
                                    : hi - ((u64)b << shift);
                else if (s.warp == 0)
                    k = max(lo, least_key_of_bin(s.bin, (uint32_t)(lo >> 32), (uint32_t)(hi >> 32), b, s.lane) << 32);
                else
                    k = b == 0 ? hi
                               : min(hi, (least_key_of_bin(s.bin, (uint32_t)(lo >> 32), (uint32_t)(hi >> 32), b - 1, s.lane)
                                          << 32) - 1);
                if (s.lane == 0) (s.warp == 0 ? sh.lo : sh.hi) = k;
            }
            if (s.tid == 0) {
                sh.bin = b;
                sh.count = bc;
                sh.above = ba;
                sh.before = b4;
                sh.target = target;
            }
        }
        __syncthreads();
        const int b = sh.bin;
        const uint32_t bc = sh.count, ba = sh.above;
        const u64 nlo = b < 0 ? lo : sh.lo, nhi = b < 0 ? 0 : sh.hi;
        before = sh.before;
        target = sh.target;
        const bool all_short = it == 0 && ba + bc <= kSampleList;
        if (b < 0 && !all_short) {
            cluster_sync_all();  // the inbox is no longer read
            return kSampleWhole;
        }
        if (all_short || bc <= kSampleList) {
            // mass above the crossing bin, for the owner search
            if (MASS && it == 0 && !all_short) {
                u64 m = 0;
                for (int i = s.tid; i < b; i += kSampleThreads) m += sh.mass[i];
                m = warp_sum(m);
                if (s.lane == 0) sh.wsum[s.warp] = m;
                __syncthreads();
                if (s.tid < (int)s.CL) {
                    m = 0;
                    for (int w = 0; w < kSampleWarps; ++w) m += sh.wsum[w];
                    st_cluster_u64(map_to_rank(smem_u32(&s.inbox[s.rank].kept), s.tid), m);
                }
            }
            const u64 from = nlo, to = all_short ? hi : nhi;
            const uint32_t counter = map_to_rank(smem_u32(&sh.list_n[slot]), 0);
#pragma unroll 4
            for (int i = s.tid; i - s.lane < s.n; i += kSampleThreads) {
                const u64 k = i < s.n ? s.composite(i) : 0;
                const bool in = i < s.n && k >= from && k <= to;
                const unsigned m = __ballot_sync(0xffffffffu, in);
                if (m) {
                    uint32_t at = 0;
                    if (s.lane == 0) at = atom_cluster_add(counter, (uint32_t)__popc(m));
                    at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << s.lane) - 1));
                    if (in && at < kSampleList) {
                        const uint32_t a = smem_u32(&sh.list[at]);
                        for (uint32_t p = 0; p < (all_short ? 1u : s.CL); ++p) st_cluster_u64(map_to_rank(a, p), k);
                    }
                }
            }
            cluster_sync_all();
            *n_list = (int)(all_short ? ba + bc : bc);
            *blo = nlo;
            *bhi = nhi;
            *before_out = before;
            *target_out = target;
            if (all_short) return kSampleShort;
            *kt = sample_list_select<MASS>(s, (int)bc, 0, false, nlo, nhi, before, target);
            *in_first = it == 0;
            return kSampleFound;
        }
        lo = nlo;
        hi = nhi;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t sample_smem[];
    SampleRow s;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(s.CL));
    s.rank = cluster_ctarank();
    s.sh = reinterpret_cast<SampleShared *>(sample_smem);
    s.inbox = reinterpret_cast<SampleInbox *>(sample_smem + sizeof(SampleShared));
    float *buf = reinterpret_cast<float *>(s.inbox + s.CL);
    s.l = buf;
    SampleShared &sh = *s.sh;
    const int tid = s.tid = threadIdx.x, warp = s.warp = tid >> 5, lane = s.lane = tid & 31;
    const uint32_t CL = s.CL, rank = s.rank;
    const int row = blockIdx.x / CL;
    if (tid < 2) sh.list_n[tid] = 0;
    pdl_wait_and_trigger();

    // this CTA's logits: NaN counts as -inf, -0 as +0; the largest, lowest index first
    const int i0 = s.i0 = min(a.V, (int)rank * a.slice);
    const int n = s.n = min(a.V, i0 + a.slice) - i0;
    const float *src = a.logits + (int64_t)row * a.ld + i0;
    u64 best = 0;
#pragma unroll 8
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
    if (lane == 0) sh.wsum[warp] = best;
    __syncthreads();
    if (tid < (int)CL) {
        best = sh.wsum[0];
        for (int w = 1; w < kSampleWarps; ++w) best = sh.wsum[w] > best ? sh.wsum[w] : best;
        st_cluster_u64(map_to_rank(smem_u32(&s.inbox[rank].best), tid), best);
    }
    cluster_sync_all();
    best = s.inbox[0].best;
    for (uint32_t p = 1; p < CL; ++p) best = s.inbox[p].best > best ? s.inbox[p].best : best;
    const float mx = key_logit((uint32_t)(best >> 32));
    float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
    if (mx == -INFINITY || !(temp > 0.f)) {  // nothing to draw from, or greedy
        if (rank == 0 && tid == 0) {
            a.token[row] = mx == -INFINITY ? -1 : (int32_t)(0xffffffffu - (uint32_t)best);
            if (a.prob) a.prob[row] = mx == -INFINITY ? 0.f : 1.f;
        }
        return;  // the whole cluster
    }
    temp = fminf(temp, 3.402823466e38f);
    s.weight = SampleWeight{mx, 46.166241308446828 / (double)temp, exp2(-lane / 32.0)};  // 32 log2(e)
    s.bin = SampleBinning{mx, (float)(128.0 / (double)temp)};

    // threshold: the weight's cut-off, then each filter raises it
    u64 kt = max(logit_key(__double2float_ru((double)mx - kSampleLive * (double)temp) + 0.f),
                 logit_key(-3.402823466e38f));
    kt <<= 32;
    u64 kmin = 0;
    const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
    if (min_p > 0.f) {
        const double c = (double)mx + (double)temp * log((double)fminf(min_p, 1.f));
        kmin = (u64)min((uint32_t)(best >> 32), logit_key(__double2float_ru(c) + 0.f)) << 32;
    }
    const int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
    const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
    float u = __ldg(a.u + row);
    u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;

    int n_list = 0, is = kSampleWhole;
    u64 blo, bhi, before, target;
    bool in_first = false, by_mass = false;
    if (top_k > 0 && top_k < a.V) {
        is = sample_filter<false>(s, kt, best, (u64)top_k, 0.0, 0, &kt, &n_list, &blo, &bhi, &before, &target, &in_first);
        in_first = false;
    }
    if (top_p < 1.f && is != kSampleShort) {
        is = sample_filter<true>(s, kt, best, 0, (double)top_p, 1, &kt, &n_list, &blo, &bhi, &before, &target, &in_first);
        by_mass = true;
    }

    if (is == kSampleShort) {  // rank 0 settles the row from its list
        if (rank != 0) return;
        if (bhi >= blo) kt = by_mass ? sample_list_select<true>(s, n_list, kt, false, blo, bhi, before, target)
                                     : sample_list_select<false>(s, n_list, kt, false, blo, bhi, before, target);
        if (!by_mass && top_p < 1.f) {
            const u64 z = sample_list_mass(s, n_list, kt);
            target = (u64)ceil((double)top_p * (double)z);
            kt = sample_list_select<true>(s, n_list, kt, false, kt, best, 0, target < 1 ? 1 : target);
        }
        kt = max(kt, kmin);
        const u64 z = sample_list_mass(s, n_list, kt);
        u64 r = (u64)((double)u * (double)z);
        if (r > z - 1) r = z - 1;
        const u64 o = sample_list_select<true>(s, n_list, kt, true, 0xffffffffu - (uint32_t)a.V, 0xffffffffu, 0, r + 1);
        for (int i = tid; i < n_list; i += kSampleThreads)
            if ((uint32_t)sh.list[i] == (uint32_t)o) {
                const double d = (double)key_logit((uint32_t)(sh.list[i] >> 32)) - (double)mx;
                a.token[row] = (int32_t)(0xffffffffu - (uint32_t)o);
                if (a.prob) a.prob[row] = (float)((d == 0.0 || isnan(d) ? 1.0 : exp(d / (double)temp)) * 8796093022208.0 / (double)z);
            }
        return;
    }

    // kept mass of every CTA
    const int seg = ((a.slice + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;  // a warp's contiguous part
    const int s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
    const bool known = in_first && kmin <= kt;  // the histogram's sums above the crossing bin, and the list's kept part
    if (!known) kt = max(kt, kmin);
    auto warp_masses = [&]() {
        u64 m = 0;
#pragma unroll 4
        for (int i = s0 + lane; i - lane < s1; i += 32) {
            const float l = i < s1 ? buf[i] : 0.f;
            const u64 w = s.weight(l);
            if (i < s1 && s.composite(i) >= kt) m += w;
        }
        m = warp_sum(m);
        if (lane == 0) sh.wsum[warp] = m;
        __syncthreads();
    };
    if (known) {
        if (tid < (int)CL) sh.tot[tid] = s.inbox[tid].kept;
        __syncthreads();
        for (int i = tid; i - lane < n_list; i += kSampleThreads) {
            const u64 e = i < n_list ? sh.list[i] : 0;
            const u64 w = s.weight(key_logit((uint32_t)(e >> 32)));
            if (i < n_list && e >= kt) atomicAdd(&sh.tot[(0xffffffffu - (uint32_t)e) / (uint32_t)a.slice], w);
        }
        __syncthreads();
    } else {
        warp_masses();
        if (tid < (int)CL) {
            u64 m = 0;
            for (int w = 0; w < kSampleWarps; ++w) m += sh.wsum[w];
            st_cluster_u64(map_to_rank(smem_u32(&s.inbox[rank].kept), tid), m);
        }
        cluster_sync_all();
        if (tid < (int)CL) sh.tot[tid] = s.inbox[tid].kept;
        __syncthreads();
    }
    // the CTA that the uniform number falls into goes on alone
    u64 z = 0, r = 0;
    {
        for (uint32_t p = 0; p < CL; ++p) z += sh.tot[p];
        r = (u64)((double)u * (double)z);
        if (r > z - 1) r = z - 1;
        uint32_t p = 0;
        while (p < CL && r >= sh.tot[p]) r -= sh.tot[p++];
        if (p != rank) return;
    }
    if (known) {
        __syncthreads();
        warp_masses();
    }
    int part = 0;  // the warp's part it falls into
    while (part < kSampleWarps - 1 && r >= sh.wsum[part]) r -= sh.wsum[part++];
    __syncthreads();
    const int per = (seg + kSampleThreads - 1) / kSampleThreads;
    const int e0 = part * seg + tid * per;
    const int e1 = min(min(n, (part + 1) * seg), e0 + per);
    u64 m = 0;
    for (int j = 0; j < per; ++j) {
        const int i = e0 + j;
        const float l = i < e1 ? buf[i] : 0.f;
        const u64 w = s.weight(l);
        if (i < e1 && s.composite(i) >= kt) m += w;
    }
    u64 inc = warp_incl_scan(m, lane);
    if (lane == 31) sh.wsum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += sh.wsum[w];
    u64 run = inc - m;
    const bool mine = run <= r && r < inc;
    if (!__ballot_sync(0xffffffffu, mine)) return;
    for (int j = 0; j < per; ++j) {
        const int i = e0 + j;
        const float l = i < e1 ? buf[i] : 0.f;
        u64 w = s.weight(l);
        if (!(i < e1 && s.composite(i) >= kt)) w = 0;
        if (mine && run <= r && r < run + w) {
            const double d = (double)l - (double)mx;
            a.token[row] = i0 + i;
            if (a.prob) a.prob[row] = (float)((l == mx ? 1.0 : exp(d / (double)temp)) * 8796093022208.0 / (double)z);
        }
        run += w;
    }
}

}  // namespace q8

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
// memory, so the logits are read once.
//   top-k: the k-th largest of the threads' own maxima bounds the k-th largest
//     element from below, closely when k is well below the number of threads.
//     A histogram of the maxima gives that bound, the few elements above it go
//     to one CTA, and it sorts them and settles the row.  Other k, and rows
//     whose large elements crowd in few threads, take a histogram of all
//     elements, and the crossing bin's elements are copied to every CTA, which
//     settles the threshold among them.
//   top-p: a histogram of counts, weighted with the bins' middles, estimates
//     the bin of the cut.  One pass then computes every weight once and sums
//     those above, in and below a window of a bin or two there, the window's
//     elements copied to every CTA; the sums show the cut in the window, or,
//     where the estimate was off, that a histogram of exact masses has to find
//     it.
// So a row takes three to six cluster barriers, the first behind the load, and at
// most one pass over its weights; only long runs of ties take more rounds.
// What bounds it is latency (barriers, scans, instructions that are fetched to
// run once) and, for top-p, the pass over the weights: 11 double operations
// each.  One B200, V = 152064, 1 / 16 / 128 rows: no filter 8 / 13 / 70 us,
// top-k 50 10 / 12 / 61, top-p 0.9 18 / 24 / 126; the logits' bytes at the
// measured 6.5 TB/s are 0.1 / 1.5 / 12 us.
#pragma once

#include "q8q8_mma.cuh"
#include "q8_device.cuh"

namespace q8 {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBins = 2048;
constexpr int kSampleGroup = 64;  // bins per group
constexpr int kSampleGroups = kSampleBins / kSampleGroup;
constexpr int kSampleList = 1024;    // a count's or an exact mass's crossing bin
constexpr int kSampleWindow = 2048;  // top-p's window
// Largest top_k of the short path.  V = 152064, 1 / 16 / 128 rows: 14 / 16 / 70 us
// at 256 there, 16 / 23 / 119 at 257 through the histogram of all elements
// (10 / 12 / 61 at 50); its list holds 512.
constexpr int kSampleShortK = 256;
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
struct alignas(16) SampleInbox {
    u64 gmass[kSampleGroups];      // a group's mass, or the bits of its fp32 estimate
    uint32_t gcnt[kSampleGroups];
    u64 best;                      // largest composite key
    u64 above, all, kept;          // masses of the pass over the weights
    uint32_t sent;                 // elements of the short list
    uint16_t pulled[kSampleGroup]; // (of this CTA's own) the bins' counts of a group in that CTA
};

struct alignas(16) SampleShared {
    // one of the two holds a list written by the cluster (top-p's window the
    // first, the others the second), the other the histogram that settles it;
    // the first is also the histogram of exact masses, read by the cluster,
    // and the sort's exchange
    u64 mass[kSampleBins];
    u64 list[kSampleList];
    uint32_t cnt[kSampleBins];  // read by the cluster
    double tab[128];            // 2^(43 - j / 128)
    u64 wsum[kSampleWarps], wabove[kSampleWarps], wall[kSampleWarps];
    u64 gm[32];                 // group sums of a list's histogram
    u64 tiny[32];
    uint32_t tiny_n;
    uint32_t span[2];           // least and largest key of a list
    uint32_t sent;              // elements this CTA has put into a list
    uint32_t short_n;           // rank 0: places of the short list given out
    // results of one thread or warp for the whole CTA
    u64 before, lo, hi, target, val;
    u64 tot[kSampleMaxCluster];
    uint32_t count, above, base;
    int bin;
};

// the logits that follow the inboxes are stored four at a time
static_assert(sizeof(SampleShared) % 16 == 0 && sizeof(SampleInbox) % 16 == 0, "the logits lie on a 16-byte boundary");
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

__device__ __forceinline__ u64 warp_max(u64 v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Where the uniform number lies in a mass of z: below 1 at the floor of u z, from
// 1 on at the last unit, which is the last kept token's however small it is.
__device__ __forceinline__ u64 sample_place(float u, u64 z) {
    const u64 r = u < 1.f ? (u64)((double)u * (double)z) : z - 1;
    return min(r, z - 1);
}

// Fixed-point weight of a logit (mx: the row's largest, finite).
// 2^(43 - (k + r) / 128) with k = round(128 log2(e) (mx - l) / T): a table of
// 2^(43 - j / 128) and the Taylor polynomial of 2^(-r / 128) to the fourth
// power (|r| <= 1/2: its remainder is below 2^-49), so 11 double operations.
// A weight below the live threshold comes out as garbage.
struct SampleWeight {
    float mx;
    double c;           // 128 log2(e) / T
    const double *tab;  // in shared memory
    __device__ __forceinline__ u64 operator()(float l) const {
        constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52
        constexpr double a = 0.0054152123481245727;    // ln 2 / 128
        const double d = (double)mx - (double)l;
        const double t = __fma_rn(d, c, kMagic);
        const int k = __double2loint(t);
        const double r = __fma_rn(d, c, -(t - kMagic));
        double p = __fma_rn(r, a * a * a * a / 24, -a * a * a / 6);
        p = __fma_rn(r, p, a * a / 2);
        p = __fma_rn(r, p, -a);
        p = __fma_rn(r, p, 1.0);
        const double w = p * tab[k & 127];
        // the exponent falls by k / 128; adding 2^52 rounds to an integer in the low bits
        const double s = __hiloint2double(__double2hiint(w) - (int)((unsigned)(k & ~127) << 13), __double2loint(w));
        return (u64)__double_as_longlong(s + 4503599627370496.0) & 0xfffffffffffffull;
    }
};

// The histogram's bins: `scale` to a unit of mx - l, the last bin takes what
// lies beyond.  Bin 0 holds the largest logits and the bin never falls as the
// logit falls: every step is a monotone fp32 operation.  Adding 2^23 rounds to
// an integer held in the low bits; the clamp takes the NaN of 0 * inf (a
// temperature whose scale overflows) to the last bin, where the row's other
// elements then are as well.
struct SampleBinning {
    float mx, scale;
    __device__ __forceinline__ float place(float l) const {  // 2^23 + the bin
        return fminf(__fmaf_rn(__fsub_rn(mx, l), scale, 8388608.f), 8388608.f + (kSampleBins - 1));
    }
    __device__ __forceinline__ int operator()(float l) const {
        return __float_as_int(place(l)) & (kSampleBins - 1);
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
    // Whether element i's composite key is at least K, l being its logit (above -inf).
    __device__ __forceinline__ bool at_least(float l, int i, float K_logit, uint32_t K_low) const {
        return l > K_logit || (l == K_logit && 0xffffffffu - (uint32_t)(i0 + i) >= K_low);
    }
    __device__ __forceinline__ u64 composite(int i) const {
        return ((u64)logit_key(l[i]) << 32) | (0xffffffffu - (uint32_t)(i0 + i));
    }
};

// 64-bit sum in shared memory as two 32-bit atomics with a carry (a 64-bit
// atomicAdd on shared memory measured four times as long).
__device__ __forceinline__ void add_mass(u64 *at, u64 w) {
    uint32_t *p = reinterpret_cast<uint32_t *>(at);
    const uint32_t lo = (uint32_t)w;
    const uint32_t hi = (uint32_t)(w >> 32) + (atomicAdd(p, lo) + lo < lo ? 1u : 0u);
    if (hi) atomicAdd(p + 1, hi);
}

// The list entry at which, in descending order, the running count (MASS: mass)
// from `before` reaches `target`.  False when that does not lie in the list.
// Whole CTA.
template <bool MASS>
__device__ bool sample_list_select(const SampleRow &s, bool window, int n, u64 before, u64 target, u64 *kt) {
    SampleShared &sh = *s.sh;
    const u64 *list = window ? sh.mass : sh.list;
    u64 *mass = window ? sh.list : sh.mass;  // 1024 bins
    uint32_t count = (uint32_t)n;
    u64 lo = 0, hi = ~0ull;
    bool first = true;
    if (count > 32) {
        // the keys it spans
        uint32_t mn = ~0u, mxv = 0;
        for (int i = s.tid; i < n; i += kSampleThreads) {
            const uint32_t k = (uint32_t)(list[i] >> 32);
            mn = min(mn, k);
            mxv = max(mxv, k);
        }
        mn = __reduce_min_sync(0xffffffffu, mn);
        mxv = __reduce_max_sync(0xffffffffu, mxv);
        if (s.tid == 0) {
            sh.span[0] = ~0u;
            sh.span[1] = 0;
        }
        for (int i = s.tid; i < 1024; i += kSampleThreads) {
            sh.cnt[i] = 0;
            if (MASS) mass[i] = 0;
        }
        __syncthreads();
        if (s.lane == 0) {
            atomicMin(&sh.span[0], mn);
            atomicMax(&sh.span[1], mxv);
        }
        __syncthreads();
        lo = (u64)sh.span[0] << 32;
        hi = (u64)sh.span[1] << 32 | 0xffffffffu;
    }
    while (count > 32) {
        const int bits = 64 - __clzll((long long)(hi - lo));
        const int shift = max(0, bits - 10);  // 1024 bins, 32 groups of 32
        if (!first) {
            for (int i = s.tid; i < 1024; i += kSampleThreads) {
                sh.cnt[i] = 0;
                if (MASS) mass[i] = 0;
            }
            __syncthreads();
        }
        for (int i = s.tid; i < n; i += kSampleThreads) {
            const u64 e = list[i];
            if (e >= lo && e <= hi) {
                const int b = (int)((hi - e) >> shift);
                atomicAdd(&sh.cnt[b], 1u);
                if (MASS) add_mass(&mass[b], s.weight(key_logit((uint32_t)(e >> 32))));
            }
        }
        __syncthreads();
        {  // group sums, two groups of 32 bins a warp (two bins a lane)
            const u64 v0 = MASS ? mass[2 * s.tid] + mass[2 * s.tid + 1] : (u64)sh.cnt[2 * s.tid] + sh.cnt[2 * s.tid + 1];
            u64 v = v0;
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if ((s.lane & 15) == 0) sh.gm[s.tid >> 4] = v;
        }
        __syncthreads();
        if (s.warp == 0) {
            u64 v = sh.gm[s.lane];
            u64 inc = before + warp_incl_scan(v, s.lane);
            const unsigned cross = __ballot_sync(0xffffffffu, inc - v < target && target <= inc);
            if (cross) {
                const int g = __ffs(cross) - 1;
                const u64 b4 = __shfl_sync(0xffffffffu, inc - v, g);
                const uint32_t c = sh.cnt[g * 32 + s.lane];
                v = MASS ? mass[g * 32 + s.lane] : c;
                inc = b4 + warp_incl_scan(v, s.lane);
                if (inc - v < target && target <= inc) {
                    const u64 top = hi - ((u64)(g * 32 + s.lane) << shift);
                    const u64 span = (1ull << shift) - 1;
                    sh.hi = top;
                    sh.lo = top - lo > span ? top - span : lo;
                    sh.before = inc - v;
                    sh.count = c;
                }
            } else if (s.lane == 0) {
                sh.count = 0;
            }
        }
        __syncthreads();
        lo = sh.lo;
        hi = sh.hi;
        before = sh.before;
        count = sh.count;
        first = false;
        __syncthreads();
        if (count == 0) return false;
    }
    if (s.tid == 0) sh.tiny_n = 0;
    __syncthreads();
    for (int i = s.tid; i < n; i += kSampleThreads) {
        const u64 e = list[i];
        if (e >= lo && e <= hi) sh.tiny[atomicAdd(&sh.tiny_n, 1u) & 31u] = e;
    }
    __syncthreads();
    if (s.warp == 0) {
        const int tn = min((int)sh.tiny_n, 32);
        const u64 e = s.lane < tn ? sh.tiny[s.lane] : 0;
        const u64 w = s.lane >= tn ? 0 : MASS ? s.weight(key_logit((uint32_t)(e >> 32))) : 1;
        u64 ex = before;
        for (int j = 0; j < tn; ++j) {
            const u64 ej = __shfl_sync(0xffffffffu, e, j), wj = __shfl_sync(0xffffffffu, w, j);
            if (ej > e) ex += wj;
        }
        const bool here = s.lane < tn && ex < target && target <= ex + w;
        if (here) sh.val = e;
        const unsigned any = __ballot_sync(0xffffffffu, here);
        if (s.lane == 0) sh.count = any;
    }
    __syncthreads();
    *kt = sh.val;
    return sh.count != 0;
}

// Histogram of the elements K in [lo, hi] (FIRST: by the logit's bin, else by
// digits of K), counts and with MASS masses.  Whole CTA.
template <bool MASS, bool FIRST>
__device__ __forceinline__ void sample_histogram(const SampleRow &s, u64 lo, u64 hi, int shift) {
    SampleShared &sh = *s.sh;
    for (int i = s.tid; i < kSampleBins; i += kSampleThreads) {
        sh.cnt[i] = 0;
        if (MASS) sh.mass[i] = 0;
    }
    __syncthreads();
    if (FIRST) {  // (hi is the row's largest)
        const float lo_l = key_logit((uint32_t)(lo >> 32));
        const uint32_t lo_w = (uint32_t)lo;
#pragma unroll 2
        for (int j = s.tid; 4 * j < s.n; j += kSampleThreads) {
            const float4 q = reinterpret_cast<const float4 *>(s.l)[j];
            const float l[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool in = s.at_least(l[c], 4 * j + c, lo_l, lo_w);
                if (in) atomicAdd(&sh.cnt[s.bin(l[c])], 1u);
                if (MASS && in) add_mass(&sh.mass[s.bin(l[c])], s.weight(l[c]));
            }
        }
    } else {
        for (int i = s.tid; i < s.n; i += kSampleThreads) {
            const u64 k = s.composite(i);
            if (k >= lo && k <= hi) {
                const int b = (int)((hi - k) >> shift);
                atomicAdd(&sh.cnt[b], 1u);
                if (MASS) add_mass(&sh.mass[b], s.weight(s.l[i]));
            }
        }
    }
    __syncthreads();
}

// The group sums of this CTA's histogram to every CTA: counts, with masses
// (MASS) or, est > 0, mass estimates exp2(-est * bin).  Four bins a thread, so
// a group is half a warp, whose lanes then each write to one CTA.  Ends with a
// cluster barrier.
template <bool MASS>
__device__ __forceinline__ void sample_share(const SampleRow &s, float est) {
    SampleShared &sh = *s.sh;
    static_assert(kSampleBins == 4 * kSampleThreads && kSampleGroup == 64 && kSampleMaxCluster == 16, "a thread's four bins");
    const uint4 q = reinterpret_cast<const uint4 *>(sh.cnt)[s.tid];
    uint32_t c = q.x + q.y + q.z + q.w;
    u64 m = 0;
    float e = 0.f;
    if (MASS)
        m = sh.mass[4 * s.tid] + sh.mass[4 * s.tid + 1] + sh.mass[4 * s.tid + 2] + sh.mass[4 * s.tid + 3];
    else if (est > 0.f) {
        const float b = 4.f * (float)s.tid;
        e = (float)q.x * exp2f(-est * b) + (float)q.y * exp2f(-est * (b + 1.f)) + (float)q.z * exp2f(-est * (b + 2.f)) +
            (float)q.w * exp2f(-est * (b + 3.f));
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
        c += __shfl_xor_sync(0xffffffffu, c, off);
        if (MASS) m += __shfl_xor_sync(0xffffffffu, m, off);
        e += __shfl_xor_sync(0xffffffffu, e, off);
    }
    const uint32_t p = s.lane & 15, g = s.tid >> 4;
    if (p < s.CL) {
        const SampleInbox *box = &s.inbox[s.rank];
        st_cluster_u32(map_to_rank(smem_u32(&box->gcnt[g]), p), c);
        if (MASS || est > 0.f) st_cluster_u64(map_to_rank(smem_u32(&box->gmass[g]), p), MASS ? m : __float_as_uint(e));
    }
    cluster_sync_all();
}

// The counts of the 64 bins of group g from all CTAs, into the inboxes' pulled.
// Whole CTA.
__device__ __forceinline__ void sample_pull_counts(const SampleRow &s, int g) {
    static_assert(kSampleThreads % kSampleGroup == 0, "a thread keeps to one bin");
    const int bin = s.tid % kSampleGroup;
#pragma unroll 1
    for (uint32_t p = s.tid / kSampleGroup; p < s.CL; p += kSampleThreads / kSampleGroup)
        s.inbox[p].pulled[bin] = (uint16_t)ld_cluster_u32(map_to_rank(smem_u32(&s.sh->cnt[g * kSampleGroup + bin]), p));
    __syncthreads();
}
// Sums of what was pulled: lane's bins 64 g + lane and + 32, of all CTAs and of
// those of lower rank.
__device__ __forceinline__ void sample_sum_counts(const SampleRow &s, uint32_t (&c)[2], uint32_t (&lower)[2]) {
    c[0] = c[1] = lower[0] = lower[1] = 0;
#pragma unroll 2
    for (uint32_t p = 0; p < s.CL; ++p) {
        const uint32_t x = s.inbox[p].pulled[s.lane], y = s.inbox[p].pulled[s.lane + 32];
        if (p == s.rank) {
            lower[0] = c[0];
            lower[1] = c[1];
        }
        c[0] += x;
        c[1] += y;
    }
}

// One filter, exactly: the threshold composite key in [lo, hi] of a count (the
// first `target`) or, MASS, of a mass (top_p of the interval's), the same in
// every CTA.  False when the filter cuts nothing.
template <bool MASS>
__device__ bool sample_filter(const SampleRow &s, u64 lo, u64 hi, u64 target, double top_p, u64 *kt) {
    SampleShared &sh = *s.sh;
    u64 before = 0;
    for (int it = 0;; ++it) {
        const int bits = 64 - __clzll((long long)(hi - lo));
        const int shift = max(0, bits - 11);     // later rounds: digits of the composite key
        if (it > 0 || MASS) cluster_sync_all();  // the last histogram and its sums are no longer read
        if (it == 0)
            sample_histogram<MASS, true>(s, lo, hi, 0);
        else
            sample_histogram<MASS, false>(s, lo, hi, shift);
        if (s.tid == 0) sh.sent = 0;
        sample_share<MASS>(s, 0.f);
        // the crossing group, then its bins from all CTAs
        int b = -1, g = -1;
        uint32_t bc = 0, off = 0;
        u64 b4 = before;
        if (s.warp == 0) {
            u64 v = 0;
#pragma unroll 2
            for (uint32_t p = 0; p < s.CL; ++p) v += MASS ? s.inbox[p].gmass[s.lane] : s.inbox[p].gcnt[s.lane];
            const u64 inc = warp_incl_scan(v, s.lane);
            const u64 all = __shfl_sync(0xffffffffu, inc, 31);
            if (MASS && it == 0) {
                target = (u64)ceil(top_p * (double)all);
                if (target < 1) target = 1;
            }
            if (target <= before + all) {
                const unsigned cross = __ballot_sync(0xffffffffu, before + inc - v < target && target <= before + inc);
                g = __ffs(cross) - 1;
                b4 = before + __shfl_sync(0xffffffffu, inc - v, g);
            }
            if (s.lane == 0) sh.bin = g;
        }
        __syncthreads();
        if (sh.bin < 0) return false;
        sample_pull_counts(s, sh.bin);
        if (s.warp == 0) {
            uint32_t fc[2], fl[2];
            u64 fm[2] = {0, 0};
            sample_sum_counts(s, fc, fl);
            if (MASS) {
#pragma unroll 4
                for (uint32_t p = 0; p < s.CL; ++p) {
                    const uint32_t am = map_to_rank(smem_u32(&sh.mass[g * kSampleGroup + s.lane]), p);
                    fm[0] += ld_cluster_u64(am);
                    fm[1] += ld_cluster_u64(am + 256);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u64 x = MASS ? fm[h] : fc[h];
                const u64 xi = b4 + warp_incl_scan(x, s.lane);
                const unsigned at = __ballot_sync(0xffffffffu, xi - x < target && target <= xi);
                if (b < 0 && at) {
                    const int f = __ffs(at) - 1;
                    b = g * kSampleGroup + 32 * h + f;
                    bc = __shfl_sync(0xffffffffu, fc[h], f);
                    off = __shfl_sync(0xffffffffu, fl[h], f);
                    b4 = __shfl_sync(0xffffffffu, xi - x, f);
                } else if (b < 0) {
                    b4 = __shfl_sync(0xffffffffu, xi, 31);
                }
            }
            if (it > 0 || bc > kSampleList) {  // the bin's keys
                const uint32_t l32 = (uint32_t)(lo >> 32), h32 = (uint32_t)(hi >> 32);
                u64 kl, kh;
                if (it > 0) {
                    kl = (hi - lo) >> shift > (u64)b ? hi - (((u64)b + 1) << shift) + 1 : lo;
                    kh = hi - ((u64)b << shift);
                } else {
                    kl = max(lo, least_key_of_bin(s.bin, l32, h32, b, s.lane) << 32);
                    kh = b == 0 ? hi : min(hi, (least_key_of_bin(s.bin, l32, h32, b - 1, s.lane) << 32) - 1);
                }
                if (s.lane == 0) {
                    sh.lo = kl;
                    sh.hi = kh;
                }
            }
            if (s.lane == 0) {
                sh.bin = b;
                sh.count = bc;
                sh.base = off;
                sh.before = b4;
                sh.target = target;
            }
        }
        __syncthreads();
        b = sh.bin;
        bc = sh.count;
        const uint32_t base = sh.base;
        before = sh.before;
        target = sh.target;
        const u64 nlo = sh.lo, nhi = sh.hi;  // (set when it > 0 or bc > kSampleList)
        if (bc <= kSampleList) {
#pragma unroll 4
            for (int i = s.tid; i < s.n; i += kSampleThreads) {
                const u64 k = s.composite(i);
                const bool in = it > 0 ? k >= nlo && k <= nhi : k >= lo && k <= hi && s.bin(s.l[i]) == b;
                if (in) {
                    const uint32_t at = base + atomicAdd(&sh.sent, 1u);
                    if (at < kSampleList)
                        for (uint32_t p = 0; p < s.CL; ++p) st_cluster_u64(map_to_rank(smem_u32(&sh.list[at]), p), k);
                }
            }
            cluster_sync_all();
            sample_list_select<MASS>(s, false, (int)bc, before, target, kt);
            return true;
        }
        lo = nlo;
        hi = nhi;
        __syncthreads();
    }
}

// Descending bitonic sort of one value a thread over the first `width` threads
// (a power of two, 32 .. kSampleThreads).  `flip`: the half of the exchange
// buffer that the next exchange writes, 0 at first and carried from one sort to
// the next: a warp may still be reading the other half.  Whole CTA.
__device__ __forceinline__ u64 sample_sort(const SampleRow &s, u64 v, int width, int &flip) {
    u64 *x = s.sh->mass;
    for (int k = 2; k <= width; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            u64 o;
            if (j >= 32) {  // two halves in turn, so one barrier a step
                x[flip + s.tid] = v;
                __syncthreads();
                o = x[flip + (s.tid ^ j)];
                flip ^= kSampleThreads;
            } else {
                o = __shfl_xor_sync(0xffffffffu, v, j);
            }
            const bool big = ((s.tid & k) == 0) == ((s.tid & j) == 0);
            v = (o > v) == big ? o : v;
        }
    return v;
}

// Inclusive sum over the threads, and the total.  Whole CTA.
__device__ __forceinline__ u64 sample_scan(const SampleRow &s, u64 v, u64 *all) {
    const u64 inc = warp_incl_scan(v, s.lane);
    __syncthreads();
    if (s.lane == 31) s.sh->wsum[s.warp] = inc;
    __syncthreads();
    const u64 x = warp_incl_scan(s.lane < kSampleWarps ? s.sh->wsum[s.lane] : 0, s.lane);
    *all = __shfl_sync(0xffffffffu, x, 31);
    const u64 b4 = __shfl_sync(0xffffffffu, x, s.warp - 1 & 31);
    return (s.warp ? b4 : 0) + inc;
}

// PER_SM: CTAs an SM is to hold (registers for one leave room for more
// elements in flight).
template <int PER_SM>
__global__ void __launch_bounds__(kSampleThreads, PER_SM) sample_kernel(const SampleArgs a) {
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
    // (the other CTAs' shared memory is theirs only once all of the cluster's have
    // started: arrived at here, waited for behind the load)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    // what no input decides; the __syncthreads behind the load publishes it
    if (tid == 0) sh.short_n = sh.sent = 0;
    for (int i = tid; i < kSampleBins; i += kSampleThreads) sh.cnt[i] = 0;
    pdl_wait_and_trigger();

    // this CTA's logits: NaN counts as -inf, -0 as +0; the largest, lowest index first
    const int i0 = s.i0 = min(a.V, (int)rank * a.slice);
    const int n = s.n = min(a.V, i0 + a.slice) - i0;
    const float *src = a.logits + (int64_t)row * a.ld + i0;
    u64 best = 0;
    {
        float mv = -INFINITY;
        int mi = 0x7fffffff;
        auto take = [&](float v, int i) {
            v += 0.f;
            if (!(v >= -INFINITY)) v = -INFINITY;
            if (v > mv || mi == 0x7fffffff) {
                mv = v;
                mi = i;
            }
            return v;
        };
        if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
            const int n4 = n >> 2;
#pragma unroll 4
            for (int j = tid; j < n4; j += kSampleThreads) {
                float4 q = __ldg(reinterpret_cast<const float4 *>(src) + j);
                q.x = take(q.x, 4 * j);
                q.y = take(q.y, 4 * j + 1);
                q.z = take(q.z, 4 * j + 2);
                q.w = take(q.w, 4 * j + 3);
                reinterpret_cast<float4 *>(buf)[j] = q;
            }
            for (int i = 4 * n4 + tid; i < n; i += kSampleThreads) buf[i] = take(__ldg(src + i), i);
        } else {
#pragma unroll 4
            for (int i = tid; i < n; i += kSampleThreads) buf[i] = take(__ldg(src + i), i);
        }
        if (tid < (-n & 3)) buf[n + tid] = -INFINITY;  // the last four are read together
        if (mi != 0x7fffffff) best = ((u64)logit_key(mv) << 32) | (0xffffffffu - (uint32_t)(i0 + mi));
    }
    const u64 own = best;  // this thread's largest
    best = warp_max(best);
    if (lane == 0) sh.wsum[warp] = best;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA has started
    __syncthreads();
    if (warp == 0) {
        best = warp_max(lane < kSampleWarps ? sh.wsum[lane] : 0);
        if (lane < (int)CL) st_cluster_u64(map_to_rank(smem_u32(&s.inbox[rank].best), lane), best);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // the row's parameters and the weight table, while the barrier completes (at
    // the kernel's start the table's exponentials delay the load of rows that wait
    // for others to end: 128 rows, mixed, 93.0 us against 91.4)
    float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
    const bool greedy = !(temp > 0.f);
    temp = fminf(temp, 3.402823466e38f);
    const double t64 = temp;
    const int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
    const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
    const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
    float u = __ldg(a.u + row);
    u = u > 0.f ? u : 0.f;
    if (tid < 128) sh.tab[tid] = 8796093022208.0 * exp2(-tid / 128.0);  // 2^43 ...
    s.weight.c = 184.66496523378733 / t64;  // 128 log2(e)
    s.weight.tab = sh.tab;
    const double min_log = min_p > 0.f ? t64 * log((double)fminf(min_p, 1.f)) : 0.0;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();  // the table, which was written behind the arrive
    best = warp_max(lane < (int)CL ? s.inbox[lane].best : 0);
    float mx = key_logit((uint32_t)(best >> 32));
    if (mx == -INFINITY || greedy) {  // nothing to draw from, or greedy
        if (rank == 0 && tid == 0) {
            a.token[row] = mx == -INFINITY ? -1 : (int32_t)(0xffffffffu - (uint32_t)best);
            if (a.prob) a.prob[row] = mx == -INFINITY ? 0.f : 1.f;
        }
        return;  // the whole cluster
    }
    u64 own_best = own;
    if (mx == INFINITY) {  // the infinite logits share the row: take them as 0 and the others as -inf
        for (int i = tid; i < n; i += kSampleThreads) buf[i] = buf[i] == INFINITY ? 0.f : -INFINITY;
        mx = 0.f;
        const u64 zero = (u64)logit_key(0.f) << 32;
        best = zero | (uint32_t)best;
        own_best = (uint32_t)(own >> 32) == logit_key(INFINITY) ? zero | (uint32_t)own : 0;
        __syncthreads();
    }
    const uint32_t key_max = (uint32_t)(best >> 32);
    s.weight.mx = s.bin.mx = mx;

    // threshold: the weight's cut-off, then each filter raises it
    u64 kt = max(logit_key(__double2float_ru((double)mx - kSampleLive * t64) + 0.f), logit_key(-3.402823466e38f));
    kt <<= 32;
    u64 kmin = 0;
    if (min_p > 0.f) kmin = (u64)min(key_max, logit_key(__double2float_ru((double)mx + min_log) + 0.f)) << 32;

    auto write = [&](uint32_t index, float l, u64 z) {
        const double w = exp(((double)l - (double)mx) / t64);
        a.token[row] = (int32_t)index;
        if (a.prob) a.prob[row] = (float)(w * 8796093022208.0 / (double)z);  // 2^43
    };

    if (top_k > 0 && top_k < a.V) {
        s.bin.scale = (float)(kSampleBins / kSampleLive / t64);  // bins over the whole live range
        if (top_k <= kSampleShortK && top_k * 4 <= (int)CL * kSampleThreads) {
            __syncthreads();
            if (own_best >= kt) atomicAdd(&sh.cnt[s.bin(key_logit((uint32_t)(own_best >> 32)))], 1u);
            __syncthreads();
            sample_share<false>(s, 0.f);
            // the bin of the k-th largest maximum, the last bin when there are fewer
            uint32_t above = 0;
            if (warp == 0) {
                uint32_t c = 0;
#pragma unroll 2
                for (uint32_t p = 0; p < CL; ++p) c += s.inbox[p].gcnt[lane];
                const uint32_t inc = warp_incl_scan(c, lane);
                const unsigned cross = __ballot_sync(0xffffffffu, inc >= (uint32_t)top_k);
                const int g = cross ? __ffs(cross) - 1 : -1;
                above = __shfl_sync(0xffffffffu, inc - c, g & 31);
                if (lane == 0) sh.bin = g;
            }
            __syncthreads();
            const int g = sh.bin;
            if (g >= 0) sample_pull_counts(s, g);
            if (warp == 0) {
                int b = kSampleBins - 1;
                if (g >= 0) {
                    uint32_t fc[2], unused[2];
                    sample_sum_counts(s, fc, unused);
                    const uint32_t c0 = above + warp_incl_scan(fc[0], lane);
                    const uint32_t c1 = __shfl_sync(0xffffffffu, c0, 31) + warp_incl_scan(fc[1], lane);
                    const unsigned at0 = __ballot_sync(0xffffffffu, c0 >= (uint32_t)top_k);
                    const unsigned at1 = __ballot_sync(0xffffffffu, c1 >= (uint32_t)top_k);
                    b = g * kSampleGroup + (at0 ? __ffs(at0) - 1 : 31 + __ffs(at1));
                }
                if (lane == 0) sh.count = (uint32_t)b;  // (with g < 0 other warps may still have to read g from sh.bin)
            }
            __syncthreads();
            // the elements down to that bin: gathered here, then sent to rank 0
            const int b = (int)sh.count;
            const float live = key_logit((uint32_t)(kt >> 32));
#pragma unroll 2
            for (int j = tid; 4 * j < n; j += kSampleThreads) {
                const float4 q = reinterpret_cast<const float4 *>(buf)[j];
                const float l[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (s.bin(l[c]) <= b && l[c] >= live) {
                        const uint32_t at = atomicAdd(&sh.sent, 1u);
                        if (at < kSampleThreads) sh.mass[at] = s.composite(4 * j + c);
                    }
            }
            __syncthreads();
            const uint32_t sent = sh.sent;
            if (tid == 0 && sent) sh.base = atom_cluster_add(map_to_rank(smem_u32(&sh.short_n), 0), sent);
            if (tid < (int)CL) st_cluster_u32(map_to_rank(smem_u32(&s.inbox[rank].sent), tid), sent);
            __syncthreads();
            if (tid < (int)sent && sh.base + tid < kSampleThreads)
                st_cluster_u64(map_to_rank(smem_u32(&sh.list[sh.base + tid]), 0), sh.mass[tid]);
            cluster_sync_all();
            uint32_t all = 0;
            for (uint32_t p = 0; p < CL; ++p) all += s.inbox[p].sent;
            if (all <= kSampleThreads) {  // rank 0 settles the row
                if (rank != 0) return;
                int width = 32, flip = 0;
                while (width < (int)all) width *= 2;
                // in the filters' order: top-k, top-p, min-p
                const u64 e = sample_sort(s, tid < (int)all ? sh.list[tid] : 0, width, flip);
                const float l = key_logit((uint32_t)(e >> 32));
                bool keep = tid < min((int)all, top_k);
                u64 w = keep ? s.weight(l) : 0, z;
                if (top_p < 1.f) {
                    const u64 inc = sample_scan(s, w, &z);
                    const u64 target = (u64)ceil((double)top_p * (double)z);
                    keep = keep && inc - w < (target < 1 ? 1 : target);
                }
                keep = keep && e >= kmin;
                // in index order: index and weight in one word (19 and 44 bits)
                const uint32_t index = 0xffffffffu - (uint32_t)e;
                const u64 y = sample_sort(s, keep ? ~((u64)index << 44 | w) : 0, width, flip);
                w = tid < width && y ? ~y & 0xfffffffffffull : 0;
                const u64 inc = sample_scan(s, w, &z);
                const u64 r = sample_place(u, z);
                if (inc - w <= r && r < inc) sh.base = (uint32_t)(~y >> 44);
                __syncthreads();
                if (keep && index == sh.base) write(index, l, z);
                return;
            }
            __syncthreads();
        }
        if (!sample_filter<false>(s, kt, best, (u64)top_k, 0.0, &kt))
            cluster_sync_all();  // the histogram's sums are no longer read
    }

    // one pass over the weights: a warp takes a contiguous part of the slice
    const int seg = ((a.slice + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
    const int s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
    const bool filter_p = top_p < 1.f;
    int w0 = kSampleBins, w1 = -1;  // window of bins
    uint32_t n_list = 0;
    if (filter_p) {
        // 128 bins to a unit: narrow where top-p cuts; they end 16 units down,
        // and a cut below that takes the exact histogram
        s.bin.scale = (float)(128.0 / t64);
        constexpr float kEst = 1.4426950408889634f / 128.f;
        sample_histogram<false, true>(s, kt, best, 0);
        if (tid == 0) sh.sent = 0;
        sample_share<false>(s, kEst);
        float b4 = 0.f, goal = 0.f;
        uint32_t ca = 0, la = 0;
        int g = 0;
        if (warp == 0) {
            float e = 0.f;
            uint32_t c = 0, low = 0;
#pragma unroll 2
            for (uint32_t p = 0; p < CL; ++p) {
                e += __uint_as_float((uint32_t)s.inbox[p].gmass[lane]);
                if (p == rank) low = c;
                c += s.inbox[p].gcnt[lane];
            }
            const float inc = warp_incl_scan(e, lane);
            const uint32_t cinc = warp_incl_scan(c, lane);
            goal = top_p * __shfl_sync(0xffffffffu, inc, 31);
            const unsigned cross = __ballot_sync(0xffffffffu, inc >= goal);
            g = cross ? __ffs(cross) - 1 : kSampleGroups - 1;
            b4 = __shfl_sync(0xffffffffu, inc - e, g);
            ca = __shfl_sync(0xffffffffu, cinc - c, g);
            la = __shfl_sync(0xffffffffu, warp_incl_scan(low, lane) - low, g);
            if (lane == 0) sh.bin = g;
        }
        __syncthreads();
        sample_pull_counts(s, sh.bin);
        if (warp == 0) {
            uint32_t fc[2], fl[2];
            sample_sum_counts(s, fc, fl);
            const int base = g * kSampleGroup;
            const float e0 = b4 + warp_incl_scan((float)fc[0] * exp2f(-kEst * (float)(base + lane)), lane);
            const float e1 = __shfl_sync(0xffffffffu, e0, 31) +
                             warp_incl_scan((float)fc[1] * exp2f(-kEst * (float)(base + 32 + lane)), lane);
            const uint32_t c0 = ca + warp_incl_scan(fc[0], lane);
            const uint32_t c1 = __shfl_sync(0xffffffffu, c0, 31) + warp_incl_scan(fc[1], lane);
            const uint32_t l0 = warp_incl_scan(fl[0], lane);
            const uint32_t l1 = __shfl_sync(0xffffffffu, l0, 31) + warp_incl_scan(fl[1], lane);
            const unsigned at0 = __ballot_sync(0xffffffffu, e0 >= goal), at1 = __ballot_sync(0xffffffffu, e1 >= goal);
            const int f = at0 ? __ffs(at0) - 1 : at1 ? 31 + __ffs(at1) : kSampleGroup - 1;
            // the estimate's bin, with the neighbour that it lies close to, within
            // the group; from the top when that is a short list
            const float ef = (float)__shfl_sync(0xffffffffu, f < 32 ? fc[0] : fc[1], f & 31) * exp2f(-kEst * (float)(base + f));
            const float part = (__shfl_sync(0xffffffffu, f < 32 ? e0 : e1, f & 31) - goal) / ef;  // of the bin, below the cut
            const int f1 = part < 0.05f ? min(f + 1, kSampleGroup - 1) : f, f0 = part > 0.95f ? max(f - 1, 0) : f;
            const uint32_t upto = __shfl_sync(0xffffffffu, f1 < 32 ? c0 : c1, f1 & 31);
            const uint32_t lower = __shfl_sync(0xffffffffu, f1 < 32 ? l0 : l1, f1 & 31);
            const uint32_t over = f0 == 0 ? ca : __shfl_sync(0xffffffffu, f0 <= 32 ? c0 : c1, (f0 - 1) & 31);
            const uint32_t lover = f0 == 0 ? 0 : __shfl_sync(0xffffffffu, f0 <= 32 ? l0 : l1, (f0 - 1) & 31);
            if (lane == 0) {
                sh.bin = upto <= kSampleWindow ? 0 : base + f0;
                sh.count = base + f1;
                sh.above = upto <= kSampleWindow ? upto : upto - over;
                sh.base = upto <= kSampleWindow ? la + lower : lower - lover;
            }
        }
        __syncthreads();
        w0 = sh.bin;
        w1 = (int)sh.count;
        n_list = sh.above;
        if (n_list > kSampleWindow) w1 = -1;  // no list: the exact histogram
    }
    // Sums of the CTA's weights K >= thr (kept); with a window also of all and
    // of those above it, its elements going to the list.
    auto masses = [&](u64 thr, bool window) {
        u64 ma = 0, mt = 0, mk = 0;
        const uint32_t base = sh.base;
        auto send = [&](uint32_t at, u64 e) {
            if (at < kSampleWindow)
                for (uint32_t p = 0; p < CL; ++p) st_cluster_u64(map_to_rank(smem_u32(&sh.mass[at]), p), e);
        };
        const float thr_l = key_logit((uint32_t)(thr >> 32)), kt_l = key_logit((uint32_t)(kt >> 32));
        const uint32_t thr_w = (uint32_t)thr, kt_w = (uint32_t)kt;
        const float first = 8388608.f + (float)w0, last = 8388608.f + (float)w1;
        const bool kept = !window || thr > kt;  // else it comes out of the other sums
#pragma unroll 1
        for (int i = s0 + 4 * lane; i < s1; i += 128) {  // four elements in flight
            const float4 q = *reinterpret_cast<const float4 *>(buf + i);
            const float l[4] = {q.x, q.y, q.z, q.w};
            u64 w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = s.weight(l[c]);
            if (kept)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (s.at_least(l[c], i + c, thr_l, thr_w)) mk += w[c];
            if (window) {
                bool live[4], in[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) live[c] = l[c] >= kt_l;
                if (kt_w)  // the threshold lies inside a run of equals
#pragma unroll
                    for (int c = 0; c < 4; ++c) live[c] = s.at_least(l[c], i + c, kt_l, kt_w);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float place = s.bin.place(l[c]);
                    if (live[c]) mt += w[c];
                    if (live[c] && place < first) ma += w[c];
                    in[c] = live[c] && place >= first && place <= last;
                }
                if (in[0] || in[1] || in[2] || in[3])
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (in[c]) {
                            const uint32_t at = atomicAdd(&sh.sent, 1u);
                            if (at < kSampleList) sh.list[at] = s.composite(i + c);  // sent below, by all threads
                            else send(base + at, s.composite(i + c));
                        }
            }
        }
        mk = warp_sum(mk);
        if (window) {
            ma = warp_sum(ma);
            mt = warp_sum(mt);
        }
        __syncthreads();
        if (lane == 0) {
            sh.wsum[warp] = mk;
            sh.wabove[warp] = ma;
            sh.wall[warp] = mt;
        }
        __syncthreads();
        if (window)
            for (int i = tid; i < (int)min(sh.sent, (uint32_t)kSampleList); i += kSampleThreads) send(base + i, sh.list[i]);
        if (warp == 0) {
            const bool in = lane < kSampleWarps;
            mk = warp_sum(in ? sh.wsum[lane] : 0);
            ma = warp_sum(in ? sh.wabove[lane] : 0);
            mt = warp_sum(in ? sh.wall[lane] : 0);
            if (lane < (int)CL) {
                const uint32_t box = map_to_rank(smem_u32(&s.inbox[rank]), lane);
                st_cluster_u64(box + offsetof(SampleInbox, kept), mk);
                st_cluster_u64(box + offsetof(SampleInbox, above), ma);
                st_cluster_u64(box + offsetof(SampleInbox, all), mt);
            }
        }
        cluster_sync_all();
    };
    // the sums over K >= thr where top-p is off, or min-p's own threshold turns out above top-p's
    u64 thr = max(kt, kmin);
    bool listed = false;  // the kept mass is that above the window and the list's kept part
    if (!filter_p || w1 >= 0) masses(thr, w1 >= 0);
    if (filter_p) {
        bool found = false;
        if (w1 >= 0) {
            const u64 above = warp_sum(lane < (int)CL ? s.inbox[lane].above : 0);
            const u64 z = warp_sum(lane < (int)CL ? s.inbox[lane].all : 0);
            u64 target = (u64)ceil((double)top_p * (double)z), cut;
            if (target < 1) target = 1;
            found = above < target && sample_list_select<true>(s, true, (int)n_list, above, target, &cut);
            if (found) kt = cut;
        }
        if (!found) {
            sample_filter<true>(s, kt, best, 0, (double)top_p, &kt);
            thr = max(kt, kmin);
            masses(thr, false);
        } else if (kt >= kmin) {
            listed = true;
            thr = kt;
        }
    }
    // kept mass of every CTA and of this one's warps
    if (tid < (int)CL) sh.tot[tid] = listed ? s.inbox[tid].above : s.inbox[tid].kept;
    if (listed && tid < kSampleWarps) sh.wsum[tid] = sh.wabove[tid];
    __syncthreads();
    if (listed) {
        for (int i = tid; i < (int)n_list; i += kSampleThreads) {
            const u64 e = sh.mass[i];  // the window's list
            if (e >= kt) {
                const u64 w = s.weight(key_logit((uint32_t)(e >> 32)));
                const uint32_t at = 0xffffffffu - (uint32_t)e, p = at / (uint32_t)a.slice;
                add_mass(&sh.tot[p], w);
                if (p == rank) add_mass(&sh.wsum[(at - i0) / seg], w);
            }
        }
        __syncthreads();
    }
    // the CTA that the uniform number falls into goes on alone
    u64 z = 0;
    for (uint32_t p = 0; p < CL; ++p) z += sh.tot[p];
    u64 r = sample_place(u, z);
    uint32_t owner = 0;
    while (owner < CL - 1 && r >= sh.tot[owner]) r -= sh.tot[owner++];
    if (owner != rank) return;
    int part = 0;  // the warp's part it falls into
    while (part < kSampleWarps - 1 && r >= sh.wsum[part]) r -= sh.wsum[part++];
    __syncthreads();
    const int per = (seg + kSampleThreads - 1) / kSampleThreads;
    const int e0 = part * seg + tid * per;
    const int e1 = min(min(n, (part + 1) * seg), e0 + per);
    u64 m = 0;
    for (int i = e0; i < e1; ++i)
        if (s.composite(i) >= thr) m += s.weight(buf[i]);
    u64 inc = warp_incl_scan(m, lane);
    if (lane == 31) sh.wsum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += sh.wsum[w];
    u64 run = inc - m;
    if (run <= r && r < inc)
        for (int i = e0; i < e1; ++i) {
            const u64 w = s.composite(i) >= thr ? s.weight(buf[i]) : 0;
            if (run <= r && r < run + w) write((uint32_t)(i0 + i), buf[i], z);
            run += w;
        }
}

}  // namespace q8

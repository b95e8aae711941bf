// lora.cuh -- low-rank adapters of many requests at once:
//   u = A_a x_n,  y_n = residual_n + scale_a B_a u,   a = adapter[n],
// A_a [R][K], B_a [M][R] (rows past the adapter's rank are not read).
//
// One thread-block cluster per token.  Its CTAs split K for u, exchange the
// partial u over distributed shared memory (added in rank order) and split M for
// B u.  Sums are fp32 in a fixed order.  The clusters of tokens that share an
// adapter each read it, through L2: all clusters run at once, so serving several
// tokens by one of them would leave the others' SMs idle (tried, up to four
// tokens a cluster: 3584 x 18944, 16 rows of one bf16 adapter of rank 128, 34 us
// against 17; 4 rows, rank 64, 13.4 against 8.0).
//
// What it reads is all it costs.  For u a warp takes 16 bytes' worth of rows of A
// (8 of two bytes, 4 of fp32) at a time and loads the next columns into registers
// while it multiplies the last: 64 KB in flight per SM.  (Rings of asynchronous
// copies in shared memory in its place, twice as deep, measured slower: what
// shared memory takes, the L1 cache lacks for loads in flight.)  B is fetched to
// L2 while u is exchanged; loading its next rows while the last are multiplied
// gave the large calls 3% and cost the small ones 4% in code.
// One B200: alone on 3584 x 18944, 16 bf16 adapters of rank 52 to 128, 23.6 us
// for 67 MB (of which the rank-128 clusters read 57 GB/s per SM for u); alone
// on 3584 x 3584, one fp32 adapter of rank 32 for 16 rows, 7.7 us, all latency:
// indices, x and A, the exchange, B.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "q8q8_mma.cuh"
#include "q8_device.cuh"

namespace q8 {

constexpr int kLoraThreads = 512;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxR = 128;
constexpr int kLoraChunk = 3328;   // most columns of x staged at a time (a multiple of 256)
constexpr int kLoraBlock = 64;     // rows of y a warp gathers before it writes them
constexpr int kLoraMaxN = 16;
constexpr int kLoraMinCluster = 4;  // the error bound's K / 128 rests on it

struct LoraArgs {
    const float *x;        // [N][K]
    const void *A;         // [n_adapters][R][K]
    const void *B;         // [n_adapters][M][R]
    const int32_t *rank;   // [n_adapters] or null (R)
    const float *scale;    // [n_adapters] or null (1)
    const int32_t *adapter;  // [N]
    const float *res;      // [N][M] or null
    float *y;              // [N][M]
    int64_t M, K;
    int N, n_adapters, R;
    int chunk;  // columns of x staged at a time: a multiple of 256, at most kLoraChunk
};

// 16 bytes that are read once: not kept in the L1 cache.
__device__ __forceinline__ ulonglong2 lora_ldg(const ulonglong2 *p) {
    ulonglong2 v;
    asm("ld.global.nc.L1::no_allocate.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "l"(p));
    return v;
}

// 8 consecutive elements of an adapter row; get(): as four fp32 pairs.
// keep(): sets the elements from the n-th on to zero, whatever they hold.
template <typename T>
struct Lora8;
template <>
struct Lora8<float> {
    ulonglong2 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = lora_ldg(reinterpret_cast<const ulonglong2 *>(p));
        b = lora_ldg(reinterpret_cast<const ulonglong2 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_ulonglong2(0, 0); }
    __device__ __forceinline__ static uint64_t first(uint64_t v, int n) {
        return n >= 2 ? v : n == 1 ? v & 0xffffffffull : 0;
    }
    __device__ __forceinline__ void keep(int n) {
        a.x = first(a.x, n);
        a.y = first(a.y, n - 2);
        b.x = first(b.x, n - 4);
        b.y = first(b.y, n - 6);
    }
    __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
        v[0] = a.x;
        v[1] = a.y;
        v[2] = b.x;
        v[3] = b.y;
    }
};
struct Lora8Short {  // two-byte elements
    uint4 q;
    __device__ __forceinline__ void load(const void *p) {
        const ulonglong2 v = lora_ldg(static_cast<const ulonglong2 *>(p));
        q = *reinterpret_cast<const uint4 *>(&v);
    }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ static uint32_t first(uint32_t v, int n) { return n >= 2 ? v : n == 1 ? v & 0xffffu : 0; }
    __device__ __forceinline__ void keep(int n) {
        q.x = first(q.x, n);
        q.y = first(q.y, n - 2);
        q.z = first(q.z, n - 4);
        q.w = first(q.w, n - 6);
    }
};
template <>
struct Lora8<__half> : Lora8Short {
    __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[i] = pack_u32x2(__float_as_uint(f.x), __float_as_uint(f.y));
        }
    }
};
template <>
struct Lora8<__nv_bfloat16> : Lora8Short {
    __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack_u32x2(w[i] << 16, w[i] & 0xffff0000u);
    }
};

__device__ __forceinline__ float lora_sum2(uint64_t v) {
    const float2 f = unpack_f32x2(v);
    return f.x + f.y;
}

// Dynamic shared memory: a chunk of x.
inline size_t lora_smem_bytes(int chunk) { return (size_t)chunk * 4; }

struct LoraShared {
    float part[kLoraMaxR];             // sums of a task: [rows of its group]
    float pu[kLoraMaxR];               // this CTA's share of u, read by the cluster
    __align__(8) float us[kLoraMaxR];  // scale u
    float ys[kLoraWarps][kLoraBlock];
};

// Halves the n values that a lane holds (the other half goes to the lane `off`
// away), so that values are summed over lanes with about one shuffle each.
template <int C>
__device__ __forceinline__ void lora_fold(float (&v)[C], int lane, int off, int n) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
        if (i < n / 2) {
            const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kLoraThreads, 1) lora_kernel(const LoraArgs a) {
    extern __shared__ __align__(16) uint8_t lora_smem[];
    __shared__ LoraShared sh;
    constexpr int ES = sizeof(T);
    constexpr int RB = 16 / ES;  // rows of A a warp takes together (what the registers hold)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t CL;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(CL));
    const uint32_t rank = cluster_ctarank();
    const int n = blockIdx.x / CL;
    pdl_wait_and_trigger();

    const float *x = a.x + n * a.K;
    const float *res = a.res ? a.res + n * a.M : nullptr;
    float *y = a.y + n * a.M;
    // this CTA's rows of y
    const int64_t m_per = (a.M + CL - 1) / CL;
    const int64_t m0 = min(a.M, m_per * rank), m1 = min(a.M, m0 + m_per);
    const int ad = __ldg(a.adapter + n);
    if (ad < 0 || ad >= a.n_adapters) {
        if (ad >= a.n_adapters && rank == 0 && tid == 0) record_error(kErrBadAdapter);
        for (int64_t m = m0 + tid; m < m1; m += kLoraThreads) y[m] = res ? res[m] : 0.f;
        return;  // the whole cluster
    }
    int r = a.R;
    if (a.rank) r = min(max(__ldg(a.rank + ad), 0), a.R);

    // u: this CTA's columns [k0, k1)
    const int64_t k_per = ((a.K / 32 + CL - 1) / CL) * 32;
    const int64_t k0 = min(a.K, k_per * rank), k1 = min(a.K, k0 + k_per);
    const T *A = static_cast<const T *>(a.A) + (int64_t)ad * a.R * a.K;
    const int groups = (r + RB - 1) / RB;
    const int ks = groups > 0 ? max(1, kLoraWarps / groups) : 1;  // warps that share a row group
    const int tasks = groups * ks;
    const int half = a.chunk / 8;
    ulonglong2 *xs = reinterpret_cast<ulonglong2 *>(lora_smem);  // [half of 8][chunk / 8]
    for (int i = tid; i < tasks * RB; i += kLoraThreads) sh.part[i] = 0.f;
    for (int64_t c0 = k0; c0 < k1; c0 += a.chunk) {
        const int units = (int)min((int64_t)a.chunk, k1 - c0) / 8;
        // unit `un` of 8 columns of a task's rows; past the last unit and the last
        // row the last ones again, whose products are not used
        const T *rows = nullptr;
        uint32_t off[RB];
        auto set_task = [&](int task) {
            const int g = task / ks;
            rows = A + (int64_t)(g * RB) * a.K + c0;
#pragma unroll
            for (int j = 0; j < RB; ++j) off[j] = (uint32_t)min(j, r - 1 - g * RB) * (uint32_t)(a.K * ES);
        };
        auto load = [&](Lora8<T>(&w)[RB], int un) {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(rows + 8 * min(un, units - 1));
#pragma unroll
            for (int j = 0; j < RB; ++j) w[j].load(reinterpret_cast<const T *>(p + off[j]));
        };
        Lora8<T> even[RB], odd[RB];
        if (warp < tasks) {  // on its way while x is staged
            set_task(warp);
            load(even, (warp % ks) * 32 + lane);
        }
        __syncthreads();  // (x of the last chunk is no longer read)
        for (int q = tid; q < units * 2; q += kLoraThreads)
            xs[(q & 1) * half + (q >> 1)] = __ldg(reinterpret_cast<const ulonglong2 *>(x + c0) + q);
        __syncthreads();
#pragma unroll 1
        for (int task = warp; task < tasks; task += kLoraWarps) {
            uint64_t acc2[RB];  // even and odd columns
#pragma unroll
            for (int j = 0; j < RB; ++j) acc2[j] = 0;
            auto multiply = [&](const Lora8<T>(&a8)[RB], int un) {
                if (un >= units) return;
                const ulonglong2 x0 = xs[un], x1 = xs[half + un];
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    uint64_t w[4];
                    a8[j].get(w);
                    acc2[j] = fma_f32x2(w[0], x0.x, acc2[j]);
                    acc2[j] = fma_f32x2(w[1], x0.y, acc2[j]);
                    acc2[j] = fma_f32x2(w[2], x1.x, acc2[j]);
                    acc2[j] = fma_f32x2(w[3], x1.y, acc2[j]);
                }
            };
            const int step = ks * 32;
            int un = (task % ks) * 32 + lane;
            if (task != warp) {
                set_task(task);
                load(even, un);
            }
#pragma unroll 1
            for (; un - lane < units; un += 2 * step) {  // two buffers in turn
                if (un - lane + step < units) load(odd, un + step);
                multiply(even, un);
                if (un - lane + 2 * step < units) load(even, un + 2 * step);
                multiply(odd, un + step);
            }
            float acc[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j) acc[j] = lora_sum2(acc2[j]);
            int off = 16, left = RB;
#pragma unroll
            for (int st = 0; st < 5; ++st, off >>= 1) {
                if (left > 1) {
                    lora_fold<RB>(acc, lane, off, left);
                    left >>= 1;
                } else {
                    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], off);
                }
            }
            // a lane holds the row whose index is its top bits
            if (lane % (32 / RB) == 0) sh.part[task * RB + lane / (32 / RB)] += acc[0];
        }
    }

    // B: a contiguous part of the CTA's rows for each warp, sent for (to L2) while
    // u is exchanged
    const int64_t w_per = (m1 - m0 + kLoraWarps - 1) / kLoraWarps;
    const int64_t w0 = min(m1, m0 + w_per * warp), w1 = min(m1, w0 + w_per);
    const T *B = static_cast<const T *>(a.B) + (int64_t)ad * a.M * a.R;
    // (a row's 128-byte lines that hold columns below the rank; short rows share lines)
    const int lines = a.R * ES > 128 ? (r * ES + 127) / 128 : 1;
    const int64_t row_step = a.R * ES > 128 ? 1 : 128 / (a.R * ES);
#pragma unroll 1
    for (int64_t m = w0 + lane * row_step; m < w1; m += 32 * row_step)
        for (int i = 0; i < lines; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(B + m * a.R + i * (128 / ES)));
    if (res)
#pragma unroll 1
        for (int64_t m = w0 + lane * 8; m < w1; m += 256) asm volatile("prefetch.global.L2 [%0];" ::"l"(res + m));

    __syncthreads();
    if (tid < r) {
        float v = 0.f;
        for (int s = 0; s < ks; ++s) v += sh.part[((tid / RB) * ks + s) * RB + tid % RB];
        sh.pu[tid] = v;
    }
    const float sc = a.scale ? __ldg(a.scale + ad) : 1.f;
    cluster_sync_all();
    if (tid < kLoraMaxR) {
        float v[16];
#pragma unroll
        for (uint32_t p = 0; p < 16; ++p)
            v[p] = p < CL && tid < r ? ld_cluster_f32(map_to_rank(smem_u32(&sh.pu[tid]), p)) : 0.f;
#pragma unroll
        for (uint32_t p = 1; p < 16; ++p) v[0] += v[p];
        sh.us[tid] = tid < r ? sc * v[0] : 0.f;  // (an infinite scale times nothing is not NaN)
    }
    // pu is not read any more; the barrier is waited for before the CTA ends
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    __syncthreads();

    const int bu = (r + 7) / 8;  // 8-column units of a row of B
    int lanes = 1;               // lanes that share a row, one unit each
    while (lanes < bu) lanes <<= 1;
    const int jc = lane & (lanes - 1), grp = lane / lanes, G = 32 / lanes;
    const int kept = min(max(r - jc * 8, 0), 8);  // what lies past the rank is not used
    uint64_t uf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) uf[i] = *reinterpret_cast<const uint64_t *>(&sh.us[jc * 8 + 2 * i]);
#pragma unroll 1
    for (int64_t m = w0; m < w1; m += kLoraBlock) {
        const int rows = (int)min((int64_t)kLoraBlock, w1 - m);
        float out[2];  // the residuals, loaded before any is stored over
#pragma unroll
        for (int h = 0; h < 2; ++h) out[h] = res && lane + 32 * h < rows ? res[m + lane + 32 * h] : 0.f;
        // (kept short: code that runs once is paid for in instruction fetches)
        constexpr int RT = 4;  // rows a lane takes together
#pragma unroll 1
        for (int j = grp; j - grp < rows; j += RT * G) {
            float v[RT];
            Lora8<T> q[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                q[i].zero();
                if (j + i * G < rows && jc < bu) q[i].load(B + (m + j + i * G) * a.R + jc * 8);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                if (kept < 8) q[i].keep(kept);
                uint64_t w[4];
                q[i].get(w);
                uint64_t s2 = mul_f32x2(w[0], uf[0]);
                s2 = fma_f32x2(w[1], uf[1], s2);
                s2 = fma_f32x2(w[2], uf[2], s2);
                s2 = fma_f32x2(w[3], uf[3], s2);
                v[i] = lora_sum2(s2);
            }
#pragma unroll 1
            for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
                for (int i = 0; i < RT; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
            if (jc == 0)
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    if (j + i * G < rows) sh.ys[warp][j + i * G] = v[i];
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < rows) y[m + lane + 32 * h] = out[h] + sh.ys[warp][lane + 32 * h];
        __syncwarp();
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace q8

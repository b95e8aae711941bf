// lora.cuh -- low-rank adapters of many requests at once:
//   u = A_a x_n,  y_n = residual_n + scale_a B_a u,   a = adapter[n],
// A_a [R][K], B_a [M][R] (rows past the adapter's rank are not read).
//
// One thread-block cluster per token; the cluster of the first of up to
// kLoraTok tokens that share an adapter serves them all, so an adapter is read
// once per kLoraTok of its tokens, and the clusters of the others leave.  The
// cluster's CTAs split K for u, exchange the partial u over distributed shared
// memory (added in rank order) and split M for B u.  Sums are fp32 in a fixed
// order.  What it reads is all it costs, so both halves keep many 16-byte loads
// in flight: a warp takes several rows of A at a time and loads the next
// columns while it multiplies the last; the first rows of B are on their way
// before u is exchanged.
#pragma once

#include <cuda_bf16.h>

#include "q8q8_mma.cuh"
#include "q8_device.cuh"

namespace q8 {

constexpr int kLoraThreads = 512;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraTok = 4;        // tokens a cluster serves
constexpr int kLoraMaxR = 128;
constexpr int kLoraChunk = 4096;   // most columns of x staged at a time (a multiple of 256)
constexpr int kLoraBRows = 8;      // rows of B a thread takes together
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

// 8 consecutive elements of an adapter row as fp32.
template <typename T>
struct Lora8;
template <>
struct Lora8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <>
struct Lora8<__half> {
    uint4 q;
    __device__ __forceinline__ void load(const __half *p) { q = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Lora8<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// x of the cluster's tokens, the halves of each 8 columns apart: [token][half][chunk / 8]
__host__ __device__ inline size_t lora_smem_bytes(int chunk) { return (size_t)kLoraTok * chunk * 4; }

struct LoraShared {
    float part[kLoraMaxR * kLoraTok * 2];  // sums of a task: [rows of its group][tokens]
    float pu[kLoraMaxR * kLoraTok];        // this CTA's share of u, read by the cluster
    float us[kLoraTok][kLoraMaxR];         // scale u
    int tok[kLoraTok];
};

// Halves the values that a lane holds at each step (the other half goes to the
// lane `off` away), so that V values are summed over the lanes with about V
// shuffles.
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

// One cluster's work for NT tokens of one adapter.  RB: rows of A a warp takes
// together.
template <typename T, int NT, int RB>
__device__ __forceinline__ void lora_cluster(const LoraArgs &a, LoraShared &sh, float4 *xs, uint32_t CL, uint32_t rank,
                                             int ad, int nt, int r) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int V = RB * NT;  // values a task sums (a power of two, at most 32)
    const int half = a.chunk / 8;
    auto xat = [&](int t, int h, int u) -> float4 & { return xs[(t * 2 + h) * half + u]; };

    // u: this CTA's columns [k0, k1)
    const int64_t k_per = ((a.K / 32 + CL - 1) / CL) * 32;
    const int64_t k0 = min(a.K, k_per * rank), k1 = min(a.K, k0 + k_per);
    const T *A = static_cast<const T *>(a.A) + (int64_t)ad * a.R * a.K;
    const int groups = (r + RB - 1) / RB;
    const int ks = groups > 0 ? max(1, kLoraWarps / groups) : 1;  // warps that share a row group
    const int tasks = groups * ks;
    for (int i = tid; i < tasks * V; i += kLoraThreads) sh.part[i] = 0.f;
    for (int64_t c0 = k0; c0 < k1; c0 += a.chunk) {
        const int units = (int)min((int64_t)a.chunk, k1 - c0) / 8;
        __syncthreads();
        for (int i = tid; i < NT * units * 2; i += kLoraThreads) {
            const int t = i / (units * 2), q = i % (units * 2);
            xat(t, q & 1, q >> 1) = t < nt ? __ldg(reinterpret_cast<const float4 *>(a.x + sh.tok[t] * a.K + c0) + q)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        for (int task = warp; task < tasks; task += kLoraWarps) {
            const int g = task / ks, s = task % ks;
            float acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
            const T *row[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j) row[j] = A + (int64_t)min(g * RB + j, r - 1) * a.K + c0;
            Lora8<T> cur[RB], nxt[RB];
            auto load = [&](Lora8<T>(&w)[RB], int un) {
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    w[j].zero();
                    if (un < units) w[j].load(row[j] + 8 * un);
                }
            };
            load(cur, s * 32 + lane);
            for (int un = s * 32 + lane; un - lane < units; un += ks * 32) {
                load(nxt, un + ks * 32);
                if (un < units) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float4 p = xat(t, 0, un), q = xat(t, 1, un);
#pragma unroll
                        for (int j = 0; j < RB; ++j) {
                            float wf[8];
                            cur[j].get(wf);
                            float &v = acc[j * NT + t];
                            v = fmaf(wf[0], p.x, v);
                            v = fmaf(wf[1], p.y, v);
                            v = fmaf(wf[2], p.z, v);
                            v = fmaf(wf[3], p.w, v);
                            v = fmaf(wf[4], q.x, v);
                            v = fmaf(wf[5], q.y, v);
                            v = fmaf(wf[6], q.z, v);
                            v = fmaf(wf[7], q.w, v);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < RB; ++j) cur[j] = nxt[j];
            }
            int off = 16, n = V;
#pragma unroll
            for (int st = 0; st < 5; ++st, off >>= 1) {
                if (n > 1) {
                    lora_fold<V>(acc, lane, off, n);
                    n >>= 1;
                } else {
                    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], off);
                }
            }
            // lane holds the value whose index is its top bits
            if (lane % (32 / V) == 0) sh.part[task * V + lane / (32 / V)] += acc[0];
        }
    }

    // the first rows of B set out before u is known
    const int64_t m_per = (((a.M + CL - 1) / CL) + 7) / 8 * 8;
    const int64_t m0 = min(a.M, m_per * rank), m1 = min(a.M, m0 + m_per);
    const int bu = (r + 7) / 8;  // 8-column units of a row of B
    int lanes = 1;               // threads that share a row
    while (lanes < bu) lanes <<= 1;
    const int jc = lane & (lanes - 1);
    const T *B = static_cast<const T *>(a.B) + (int64_t)ad * a.M * a.R + jc * 8;
    const int64_t step = (int64_t)kLoraThreads / lanes * kLoraBRows;
    int64_t mb = m0 + (int64_t)(tid / lanes) * kLoraBRows;
    Lora8<T> w[kLoraBRows];
    auto load_b = [&](int64_t m) {
#pragma unroll
        for (int j = 0; j < kLoraBRows; ++j) {
            w[j].zero();
            if (m + j < m1 && jc < bu) w[j].load(B + (m + j) * a.R);
        }
    };
    load_b(mb);

    __syncthreads();
    for (int i = tid; i < r * NT; i += kLoraThreads) {
        const int j = i / NT, t = i % NT;
        float v = 0.f;
        for (int s = 0; s < ks; ++s) v += sh.part[((j / RB) * ks + s) * V + (j % RB) * NT + t];
        sh.pu[i] = v;
    }
    cluster_sync_all();
    const float sc = a.scale ? __ldg(a.scale + ad) : 1.f;
    for (int i = tid; i < kLoraMaxR * NT; i += kLoraThreads) {
        float v[16];
#pragma unroll
        for (uint32_t p = 0; p < 16; ++p)
            v[p] = p < CL && i < r * NT ? ld_cluster_f32(map_to_rank(smem_u32(&sh.pu[i]), p)) : 0.f;
#pragma unroll
        for (uint32_t p = 1; p < 16; ++p) v[0] += v[p];
        sh.us[i % NT][i / NT] = sc * v[0];
    }
    // pu is not read after this barrier completes; it is waited for at the end
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    __syncthreads();

    float uf[NT][8];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) uf[t][i] = sh.us[t][jc * 8 + i];
    const int64_t rounds = m1 > m0 ? (m1 - m0 + step - 1) / step : 0;
    for (int64_t it = 0; it < rounds; ++it, mb += step) {
        constexpr int VB = kLoraBRows * NT;
        float v[VB];
#pragma unroll
        for (int j = 0; j < kLoraBRows; ++j) {
            float wf[8];
            w[j].get(wf);
#pragma unroll
            for (int t = 0; t < NT; ++t) v[j * NT + t] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float b = jc * 8 + i < r ? wf[i] : 0.f;  // what lies past the rank is not used
#pragma unroll
                for (int t = 0; t < NT; ++t) v[j * NT + t] = fmaf(b, uf[t][i], v[j * NT + t]);
            }
        }
        if (it + 1 < rounds) load_b(mb + step);
        // sum over the row's threads
        int n = VB, at = 0;
        bool mine = true;
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            const int off = lanes >> (st + 1);
            if (off > 0) {
                if (VB >> st > 1) {
                    lora_fold<VB>(v, lane, off, VB >> st);
                    if (lane & off) at += VB >> (st + 1);
                    n = VB >> (st + 1);
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
                    mine = mine && !(lane & off);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VB; ++i)
            if (i < n && mine) {
                const int t = (at + i) % NT;
                const int64_t m = mb + (at + i) / NT;
                if (t < nt && m < m1) {
                    const int64_t o = sh.tok[t] * a.M + m;
                    a.y[o] = (a.res ? a.res[o] : 0.f) + v[i];
                }
            }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
__global__ void __launch_bounds__(kLoraThreads, 1) lora_kernel(const LoraArgs a) {
    extern __shared__ __align__(16) uint8_t lora_smem[];
    __shared__ LoraShared sh;
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t CL;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(CL));
    const uint32_t rank = cluster_ctarank();
    const int n = blockIdx.x / CL;
    pdl_wait_and_trigger();

    // which tokens this cluster serves
    const int mine = lane < a.N ? __ldg(a.adapter + lane) : -1;
    const int ad = __shfl_sync(0xffffffffu, mine, n);
    if (ad < 0 || ad >= a.n_adapters) {
        if (ad >= a.n_adapters && rank == 0 && tid == 0) record_error(kErrBadAdapter);
        const int64_t m_per = (a.M + CL - 1) / CL;
        const int64_t m0 = min(a.M, m_per * rank), m1 = min(a.M, m0 + m_per);
        for (int64_t m = m0 + tid; m < m1; m += kLoraThreads)
            a.y[n * a.M + m] = a.res ? a.res[n * a.M + m] : 0.f;
        return;  // the whole cluster
    }
    unsigned same = __ballot_sync(0xffffffffu, lane < a.N && mine == ad);
    if (__popc(same & ((1u << n) - 1)) % kLoraTok != 0) return;  // the whole cluster: another one serves it
    same &= ~((1u << n) - 1);
    const int nt = min(__popc(same), kLoraTok);
#pragma unroll
    for (int i = 0; i < kLoraTok; ++i) {
        if (tid == 0) sh.tok[i] = same ? __ffs(same) - 1 : n;
        same &= same - 1;
    }
    __syncthreads();
    int r = a.R;
    if (a.rank) r = min(max(__ldg(a.rank + ad), 0), a.R);
    float4 *xs = reinterpret_cast<float4 *>(lora_smem);
    // fp32 rows take twice the registers
    constexpr int RB = sizeof(T) == 4 ? 4 : 8;
    if (nt == 1)
        lora_cluster<T, 1, RB>(a, sh, xs, CL, rank, ad, nt, r);
    else if (nt == 2)
        lora_cluster<T, 2, RB>(a, sh, xs, CL, rank, ad, nt, r);
    else
        lora_cluster<T, 4, 4>(a, sh, xs, CL, rank, ad, nt, r);
}

}  // namespace q8

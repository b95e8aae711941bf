// lora.cuh -- low-rank adapters of many requests at once:
//   u = A_a x_n,  y_n = residual_n + scale_a B_a u,   a = adapter[n],
// A_a [R][K], B_a [M][R] (rows past the adapter's rank are not read).
//
// One thread-block cluster per token; the cluster of the first of up to
// kLoraTok tokens that share an adapter serves them all, so an adapter is read
// once per kLoraTok of its tokens, and the clusters of the others leave.  The
// cluster's CTAs split K for u, exchange the partial u over distributed shared
// memory (added in rank order) and split M for B u.  Sums are fp32 in a fixed
// order.
#pragma once

#include <cuda_bf16.h>

#include "q8q8_mma.cuh"
#include "q8_device.cuh"

namespace q8 {

constexpr int kLoraThreads = 512;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraTok = 4;        // tokens a cluster serves
constexpr int kLoraMaxR = 128;
constexpr int kLoraRows = 4;       // rows of A a warp takes together
constexpr int kLoraChunk = 2048;   // columns of x staged at a time (a multiple of 256)
constexpr int kLoraMaxN = 16;

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

template <typename T>
__global__ void __launch_bounds__(kLoraThreads, 1) lora_kernel(const LoraArgs a) {
    __shared__ float4 xs[kLoraTok][2][kLoraChunk / 8];  // x, the halves of each 8 columns apart
    __shared__ float part[2 * kLoraMaxR / kLoraRows][kLoraRows * kLoraTok];  // a task's sums
    __shared__ float pu[kLoraMaxR * kLoraTok];                     // this CTA's share of u, read by the cluster
    __shared__ float us[kLoraTok][kLoraMaxR];                      // scale u
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t CL;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(CL));
    const uint32_t rank = cluster_ctarank();
    const int n = blockIdx.x / CL;
    pdl_wait_and_trigger();

    // which tokens this cluster serves
    const int mine = lane < a.N ? __ldg(a.adapter + lane) : -1;
    const int ad = __shfl_sync(0xffffffffu, mine, n);
    const int64_t m_per = (a.M + CL - 1) / CL;
    const int64_t m0 = min(a.M, m_per * rank), m1 = min(a.M, m0 + m_per);
    if (ad < 0 || ad >= a.n_adapters) {
        if (ad >= a.n_adapters && rank == 0 && tid == 0) record_error(kErrBadAdapter);
        for (int64_t m = m0 + tid; m < m1; m += kLoraThreads)
            a.y[n * a.M + m] = a.res ? a.res[n * a.M + m] : 0.f;
        return;  // the whole cluster
    }
    unsigned same = __ballot_sync(0xffffffffu, lane < a.N && mine == ad);
    if (__popc(same & ((1u << n) - 1)) % kLoraTok != 0) return;  // the whole cluster: another one serves it
    same &= ~((1u << n) - 1);
    __shared__ int tok_s[kLoraTok];
    int tok[kLoraTok];
    int nt = 0;
#pragma unroll
    for (int i = 0; i < kLoraTok; ++i) {
        tok[i] = same ? __ffs(same) - 1 : n;
        nt += same ? 1 : 0;
        same &= same - 1;
        if (tid == 0) tok_s[i] = tok[i];
    }
    int r = a.R;
    if (a.rank) r = min(max(__ldg(a.rank + ad), 0), a.R);

    // u: this CTA's columns [k0, k1)
    const int64_t k_per = ((a.K / 32 + CL - 1) / CL) * 32;
    const int64_t k0 = min(a.K, k_per * rank), k1 = min(a.K, k0 + k_per);
    const T *A = static_cast<const T *>(a.A) + (int64_t)ad * a.R * a.K;
    const int groups = (r + kLoraRows - 1) / kLoraRows;
    const int ks = groups > 0 ? max(1, kLoraWarps / groups) : 1;  // warps that share a row group
    for (int i = tid; i < groups * ks * kLoraRows * kLoraTok; i += kLoraThreads)
        part[i / (kLoraRows * kLoraTok)][i % (kLoraRows * kLoraTok)] = 0.f;
    for (int64_t c0 = k0; c0 < k1; c0 += kLoraChunk) {
        const int cols = (int)min((int64_t)kLoraChunk, k1 - c0);
        __syncthreads();
        for (int i = tid; i < kLoraTok * (cols / 4); i += kLoraThreads) {
            const int t = i / (cols / 4), q = i % (cols / 4);
            xs[t][q & 1][q >> 1] = t < nt ? *reinterpret_cast<const float4 *>(a.x + tok_s[t] * a.K + c0 + 4 * q)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        for (int task = warp; task < groups * ks; task += kLoraWarps) {
            const int g = task / ks, s = task % ks;
            float acc[kLoraRows * kLoraTok];
#pragma unroll
            for (int i = 0; i < kLoraRows * kLoraTok; ++i) acc[i] = 0.f;
            const T *row = A + (int64_t)(g * kLoraRows) * a.K + c0;
#pragma unroll 2
            for (int un = s * 32 + lane; un < cols / 8; un += ks * 32) {
                Lora8<T> w[kLoraRows];
#pragma unroll
                for (int j = 0; j < kLoraRows; ++j) {
                    if (g * kLoraRows + j < r)
                        w[j].load(row + j * a.K + 8 * un);
                    else
                        w[j].zero();
                }
                float wf[kLoraRows][8];
#pragma unroll
                for (int j = 0; j < kLoraRows; ++j) w[j].get(wf[j]);
#pragma unroll
                for (int t = 0; t < kLoraTok; ++t) {
                    const float4 p = xs[t][0][un], q = xs[t][1][un];
#pragma unroll
                    for (int j = 0; j < kLoraRows; ++j) {
                        float &v = acc[j * kLoraTok + t];
                        v = fmaf(wf[j][0], p.x, v);
                        v = fmaf(wf[j][1], p.y, v);
                        v = fmaf(wf[j][2], p.z, v);
                        v = fmaf(wf[j][3], p.w, v);
                        v = fmaf(wf[j][4], q.x, v);
                        v = fmaf(wf[j][5], q.y, v);
                        v = fmaf(wf[j][6], q.z, v);
                        v = fmaf(wf[j][7], q.w, v);
                    }
                }
            }
            // warp sums of the 16 values: halve the values held at each step
#pragma unroll
            for (int h = 8, off = 16; h >= 1; h >>= 1, off >>= 1) {
                const bool up = lane & off;
#pragma unroll
                for (int i = 0; i < h; ++i) {
                    const float send = up ? acc[i] : acc[i + h];
                    const float keep = up ? acc[i + h] : acc[i];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                }
            }
            acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
            if (!(lane & 1)) part[task][lane >> 1] += acc[0];
        }
    }
    __syncthreads();
    for (int i = tid; i < r * kLoraTok; i += kLoraThreads) {
        const int j = i / kLoraTok, t = i % kLoraTok;
        float v = 0.f;
        for (int s = 0; s < ks; ++s) v += part[(j / kLoraRows) * ks + s][(j % kLoraRows) * kLoraTok + t];
        pu[i] = v;
    }
    cluster_sync_all();
    const float sc = a.scale ? __ldg(a.scale + ad) : 1.f;
    for (int i = tid; i < kLoraMaxR * kLoraTok; i += kLoraThreads) {
        float v = 0.f;
        if (i < r * kLoraTok)
            for (uint32_t p = 0; p < CL; ++p) v += ld_cluster_f32(map_to_rank(smem_u32(&pu[i]), p));
        us[i % kLoraTok][i / kLoraTok] = sc * v;
    }
    __syncthreads();

    // y: this CTA's rows; `lanes` threads share a row, 8 columns of B each
    const int units = (r + 7) / 8;
    int lanes = 1;
    while (lanes < units) lanes <<= 1;
    const int jc = lane & (lanes - 1);
    float uf[kLoraTok][8];
#pragma unroll
    for (int t = 0; t < kLoraTok; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) uf[t][i] = us[t][jc * 8 + i];
    const T *B = static_cast<const T *>(a.B) + (int64_t)ad * a.M * a.R;
    const int per = kLoraThreads / lanes;
    const int64_t passes = (m1 - m0 + per - 1) / per;
    for (int64_t it = 0; it < passes; ++it) {
        const int64_t m = m0 + it * per + tid / lanes;
        float v[kLoraTok] = {0.f, 0.f, 0.f, 0.f};
        if (m < m1 && jc < units) {
            Lora8<T> w;
            w.load(B + m * a.R + jc * 8);
            float wf[8];
            w.get(wf);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float b = jc * 8 + i < r ? wf[i] : 0.f;
#pragma unroll
                for (int t = 0; t < kLoraTok; ++t) v[t] = fmaf(b, uf[t][i], v[t]);
            }
        }
        for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
            for (int t = 0; t < kLoraTok; ++t) v[t] += __shfl_xor_sync(0xffffffffu, v[t], off);
        if (m < m1 && jc == 0) {
#pragma unroll
            for (int t = 0; t < kLoraTok; ++t)
                if (t < nt) {
                    const int64_t o = tok[t] * a.M + m;
                    a.y[o] = (a.res ? a.res[o] : 0.f) + v[t];
                }
        }
    }
    cluster_sync_all();  // pu is read by the whole cluster
}

}  // namespace q8

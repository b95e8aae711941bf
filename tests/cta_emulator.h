// cta_emulator.h -- runs one cluster of a CUDA kernel on the CPU: a fiber per
// thread, warp operations, __syncthreads, cluster barriers and shared memory of
// other CTAs.  Threads are switched at these operations only, and which warp
// goes on is the caller's choice, so a schedule can let one warp run as far
// ahead of the others as the kernel's barriers allow.  What the barriers do not
// order then comes out wrong, deterministically: as another result, as an
// access out of range, as warps that wait at different barriers.
// Compiled by g++ with the kernel's source behind it (tests/sample_emulator.py).
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <sys/mman.h>
#include <ucontext.h>

#include <algorithm>
#include <type_traits>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)

struct alignas(16) float4 { float x, y, z, w; };
struct alignas(16) uint4 { uint32_t x, y, z, w; };

namespace emu {

enum State { kRun, kWarp, kCta, kCluster, kDone };
constexpr size_t kStack = 64 << 10;
constexpr size_t kGuard = 4 << 10;

struct Fiber {
    ucontext_t ctx;
    int cta, tid;
    State state;
    int arrived;  // cluster barriers arrived at and not yet waited for
    long phase;   // cluster barriers waited for
};
struct Warp {
    uint64_t val[2][32];
    int par = 0, count = 0;
};
struct Cluster {
    int ctas, threads, row;
    std::vector<Fiber> f;
    std::vector<Warp> w;
    std::vector<std::vector<uint8_t>> smem;
    std::vector<int> cta_count, cta_alive, order;
    size_t smem_bytes;
    int cl_count, alive;
    long cl_phase;
    ucontext_t main;
    Fiber *cur;
    void (*body)(const void *);
    const void *args;
    char err[256];
    uint32_t rng;  // 0: the fixed order, else a random one at every switch
};
inline Cluster *g;

inline void yield() { swapcontext(&g->cur->ctx, &g->main); }
[[noreturn]] inline void fail(const char *what, long a = 0, long b = 0) {
    snprintf(g->err, sizeof g->err, "CTA %d thread %d: %s (%ld, %ld)", g->cur->cta, g->cur->tid, what, a, b);
    setcontext(&g->main);
    abort();
}
inline Warp &warp() { return g->w[(g->cur->cta * g->threads + g->cur->tid) / 32]; }

// All 32 lanes give a value and read the others'.
inline const uint64_t *exchange(uint64_t v) {
    Warp &w = warp();
    const int par = w.par;
    w.val[par][g->cur->tid & 31] = v;
    if (++w.count == 32) {
        w.count = 0;
        w.par ^= 1;
        Fiber *f = &g->f[(g->cur->cta * g->threads + g->cur->tid) & ~31];
        for (int i = 0; i < 32; ++i) f[i].state = kRun;
    } else {
        g->cur->state = kWarp;
        yield();
    }
    return w.val[par];
}

inline void cta_release(int cta) {
    if (g->cta_count[cta] == 0 || g->cta_count[cta] != g->cta_alive[cta]) return;
    g->cta_count[cta] = 0;
    for (int i = 0; i < g->threads; ++i) {
        Fiber &f = g->f[cta * g->threads + i];
        if (f.state == kCta) f.state = kRun;
    }
}
inline void cluster_release() {
    if (g->cl_count == 0 || g->cl_count != g->alive) return;
    g->cl_count = 0;
    ++g->cl_phase;
    for (Fiber &f : g->f)
        if (f.state == kCluster) f.state = kRun;
}

inline void sync_cta() {
    ++g->cta_count[g->cur->cta];
    g->cur->state = kCta;
    cta_release(g->cur->cta);
    yield();
}
inline void cluster_arrive() {
    if (g->cur->arrived++) fail("arrives at the cluster barrier twice without a wait");
    ++g->cl_count;
    cluster_release();
    yield();  // whoever is ahead goes on first
}
inline void cluster_wait() {
    if (!g->cur->arrived--) fail("waits at the cluster barrier without an arrive");
    if (g->cl_phase == g->cur->phase) {
        g->cur->state = kCluster;
        yield();
    }
    ++g->cur->phase;
}

// An address in the cluster's shared memory: 1 + the CTA above bit 24, its offset below.
inline uint32_t address(const void *p) {
    const uint8_t *b = g->smem[g->cur->cta].data() + kGuard, *q = static_cast<const uint8_t *>(p);
    if (q < b || q >= b + g->smem_bytes) fail("address outside its own shared memory", q - b, (long)g->smem_bytes);
    return (uint32_t)(g->cur->cta + 1) << 24 | (uint32_t)(q - b);
}
inline uint32_t map_rank(uint32_t a, uint32_t rank) {
    if (rank >= (uint32_t)g->ctas) fail("rank past the cluster", rank);
    return (rank + 1) << 24 | (a & 0xffffffu);
}
inline void *at(uint32_t a, size_t size) {
    const int cta = (int)(a >> 24) - 1;
    const size_t off = a & 0xffffffu;
    if (cta < 0 || cta >= g->ctas || off + size > g->smem_bytes || off % size) fail("bad shared-memory address", cta, (long)off);
    if (cta != g->cur->cta && g->cur->phase == 0) fail("access to another CTA before any cluster barrier", cta);
    if (cta != g->cur->cta && g->cta_alive[cta] == 0) fail("access to a CTA that has ended", cta);
    return g->smem[cta].data() + kGuard + off;
}

inline void entry() {
    g->body(g->args);
    Fiber *f = g->cur;
    f->state = kDone;
    --g->cta_alive[f->cta];
    --g->alive;
    if (f->arrived) fail("ends with a cluster barrier not waited for");
    cta_release(f->cta);
    cluster_release();
    setcontext(&g->main);
}

// order: the warps' precedence (index cta * warps + warp).  fill: the byte that
// shared memory holds at the start.  Empty string: ended well.
inline const char *run(Cluster &c, int row, int ctas, int threads, size_t smem, const int *order, uint32_t rng, int fill,
                       void (*body)(const void *), const void *args) {
    static uint8_t *stacks = nullptr;
    static size_t have = 0;
    const size_t n = (size_t)ctas * threads;
    if (n > have) {
        stacks = static_cast<uint8_t *>(mmap(nullptr, n * kStack, PROT_READ | PROT_WRITE,
                                             MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
        have = n;
    }
    g = &c;
    c.ctas = ctas, c.threads = threads, c.row = row, c.smem_bytes = smem;
    c.f.resize(n);
    c.w.assign(n / 32, Warp());
    c.smem.assign(ctas, std::vector<uint8_t>(smem + 2 * kGuard, (uint8_t)fill));
    c.cta_count.assign(ctas, 0);
    c.cta_alive.assign(ctas, threads);
    c.order.assign(order, order + n / 32);
    c.cl_count = 0, c.alive = (int)n, c.cl_phase = 0;
    c.body = body, c.args = args, c.rng = rng;
    c.err[0] = 0;
    for (size_t i = 0; i < n; ++i) {
        Fiber &f = c.f[i];
        f.cta = (int)(i / threads), f.tid = (int)(i % threads), f.state = kRun, f.arrived = 0, f.phase = 0;
        getcontext(&f.ctx);
        f.ctx.uc_stack.ss_sp = stacks + i * kStack;
        f.ctx.uc_stack.ss_size = kStack;
        f.ctx.uc_link = nullptr;
        makecontext(&f.ctx, reinterpret_cast<void (*)()>(entry), 0);
    }
    while (c.alive > 0 && !c.err[0]) {
        Fiber *next = nullptr;
        size_t from = 0;
        if (c.rng) {
            c.rng = c.rng * 1664525u + 1013904223u;
            from = (c.rng >> 8) % c.order.size();
        }
        for (size_t k = 0; k < c.order.size() && !next; ++k) {
            Fiber *f = &c.f[c.order[(from + k) % c.order.size()] * 32];
            for (int i = 0; i < 32 && !next; ++i)
                if (f[i].state == kRun) next = f + i;
        }
        if (!next) {
            int at[5] = {0, 0, 0, 0, 0};
            for (const Fiber &f : c.f) ++at[f.state];
            snprintf(c.err, sizeof c.err, "threads wait for good: %d for their warp, %d at __syncthreads, %d at the cluster barrier, %d ended",
                     at[kWarp], at[kCta], at[kCluster], at[kDone]);
            break;
        }
        c.cur = next;
        swapcontext(&c.main, &next->ctx);
    }
    if (!c.err[0])
        for (int r = 0; r < ctas; ++r)
            for (size_t i = 0; i < kGuard; ++i)
                if (c.smem[r][i] != (uint8_t)fill || c.smem[r][kGuard + smem + i] != (uint8_t)fill)
                    snprintf(c.err, sizeof c.err, "CTA %d wrote outside its shared memory", r);
    return c.err;
}

struct Index {
    int cta;
    operator int() const { return cta ? g->row * g->ctas + g->cur->cta : g->cur->tid; }
};
struct Dim {
    Index x;
};
inline uint8_t *smem() { return g->smem[g->cur->cta].data() + kGuard; }

template <typename T>
uint64_t bits(T v) {
    uint64_t b = 0;
    memcpy(&b, &v, sizeof v);
    return b;
}
template <typename T>
T value(uint64_t b) {
    T v;
    memcpy(&v, &b, sizeof v);
    return v;
}
template <typename To, typename From>
To cast(From v) {
    To t;
    static_assert(sizeof t == sizeof v, "");
    memcpy(&t, &v, sizeof t);
    return t;
}

}  // namespace emu

static const emu::Dim threadIdx = {{0}}, blockIdx = {{1}};

template <typename T>
T __shfl_sync(unsigned, T v, int lane) { return emu::value<T>(emu::exchange(emu::bits(v))[lane & 31]); }
template <typename T>
T __shfl_xor_sync(unsigned, T v, int mask) { return emu::value<T>(emu::exchange(emu::bits(v))[(emu::g->cur->tid ^ mask) & 31]); }
template <typename T>
T __shfl_up_sync(unsigned, T v, int by) {
    const int lane = emu::g->cur->tid & 31;
    return emu::value<T>(emu::exchange(emu::bits(v))[lane >= by ? lane - by : lane]);
}
inline unsigned __ballot_sync(unsigned, bool p) {
    const uint64_t *v = emu::exchange(p);
    unsigned m = 0;
    for (int i = 0; i < 32; ++i) m |= (unsigned)v[i] << i;
    return m;
}
inline unsigned __reduce_min_sync(unsigned, unsigned x) {
    const uint64_t *v = emu::exchange(x);
    return (unsigned)*std::min_element(v, v + 32);
}
inline unsigned __reduce_max_sync(unsigned, unsigned x) {
    const uint64_t *v = emu::exchange(x);
    return (unsigned)*std::max_element(v, v + 32);
}
inline void __syncthreads() { emu::sync_cta(); }
inline void __syncwarp() { emu::exchange(0); }

template <typename T>
T __ldg(const T *p) { return *p; }
inline uint32_t atomicAdd(uint32_t *p, uint32_t v) { const uint32_t o = *p; *p += v; return o; }
inline uint32_t atomicMin(uint32_t *p, uint32_t v) { const uint32_t o = *p; *p = std::min(o, v); return o; }
inline uint32_t atomicMax(uint32_t *p, uint32_t v) { const uint32_t o = *p; *p = std::max(o, v); return o; }

template <typename A, typename B>
typename std::common_type<A, B>::type min(A a, B b) {
    const typename std::common_type<A, B>::type x = a, y = b;
    return x < y ? x : y;
}
template <typename A, typename B>
typename std::common_type<A, B>::type max(A a, B b) {
    const typename std::common_type<A, B>::type x = a, y = b;
    return x > y ? x : y;
}
inline int __ffs(unsigned v) { return __builtin_ffs((int)v); }
inline int __clzll(long long v) { return v ? __builtin_clzll((unsigned long long)v) : 64; }
inline uint32_t __float_as_uint(float v) { return emu::cast<uint32_t>(v); }
inline int __float_as_int(float v) { return emu::cast<int>(v); }
inline float __uint_as_float(uint32_t v) { return emu::cast<float>(v); }
inline float __fmaf_rn(float a, float b, float c) { return fmaf(a, b, c); }
inline float __fsub_rn(float a, float b) { return a - b; }
inline double __fma_rn(double a, double b, double c) { return fma(a, b, c); }
inline int __double2loint(double v) { return (int)(uint32_t)emu::bits(v); }
inline int __double2hiint(double v) { return (int)(uint32_t)(emu::bits(v) >> 32); }
inline double __hiloint2double(int hi, int lo) { return emu::value<double>((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo); }
inline long long __double_as_longlong(double v) { return (long long)emu::bits(v); }
inline float __double2float_ru(double v) {
    const float f = (float)v;
    return (double)f < v ? nextafterf(f, INFINITY) : v < 0 && f == -INFINITY && v > -INFINITY ? -3.402823466e38f : f;
}

// the library's wrappers of instructions that have no C++ form
namespace q8 {
inline uint32_t smem_u32(const void *p) { return emu::address(p); }
inline uint32_t map_to_rank(uint32_t a, uint32_t rank) { return emu::map_rank(a, rank); }
inline uint32_t cluster_ctarank() { return (uint32_t)emu::g->cur->cta; }
inline void cluster_sync_all() {
    emu::cluster_arrive();
    emu::cluster_wait();
}
inline void pdl_wait_and_trigger() {}
}  // namespace q8

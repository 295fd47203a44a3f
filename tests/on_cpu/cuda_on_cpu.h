// cuda_on_cpu.h -- enough of CUDA's device language to compile and run a kernel's source as
// plain C++: a CUDA thread is a fiber, blocks run one after another, the blocks of a cluster
// together.  Every warp operation, and every barrier, is a point that all threads of its mask have
// to reach; a fiber runs undisturbed from one to the next.
#pragma once
#undef _FORTIFY_SOURCE               // its longjmp stays on one stack
#include <setjmp.h>
#include <ucontext.h>

#include <algorithm>
#include <bit>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <memory>
#include <type_traits>
#include <vector>

#define __device__
#define __global__
#define __forceinline__ inline
#define __noinline__
#define __shared__ static
#define __launch_bounds__(...)
#define __align__(x) alignas(x)

using std::max;
using std::min;
inline int64_t min(int64_t a, int b) { return a < b ? a : b; }

// ------------------------------------------------------------------- fibers
struct Barrier {
    int threads = 0, arrived = 0;
    unsigned turn = 0;
};
struct Warp {
    Barrier meet;
    uint64_t value[32];
};
struct Cta {
    std::unique_ptr<char[]> space;      // dynamic shared memory, with room to align
    char* dynamic = nullptr;
    Barrier all;
    std::vector<Warp> warps;
    int count = 0, rank = 0;
    struct Cluster* cluster = nullptr;
};
struct Cluster {
    std::vector<Cta> ctas;
    Barrier all;
};
struct Dim { unsigned x, y, z; };
struct Fiber {
    ucontext_t begin;
    jmp_buf go_on;
    Dim thread;
    Cta* cta;
    bool begun = false, done = false;
};
inline Fiber* g_fiber;
inline jmp_buf g_scheduler;
inline const std::function<void()>* g_kernel;
inline Dim g_block, gridDim{1, 1, 1};
#define threadIdx (g_fiber->thread)
#define blockIdx (g_blocks())
inline Dim g_blocks() { return {g_block.x + (unsigned)g_fiber->cta->rank, 0, 0}; }

inline void reach(Barrier& b) {
    const unsigned turn = b.turn;
    if (++b.arrived == b.threads) {
        b.arrived = 0;
        ++b.turn;
        return;
    }
    Fiber* const mine = g_fiber;
    while (b.turn == turn)
        if (!_setjmp(mine->go_on)) _longjmp(g_scheduler, 1);
}
inline void fiber_main() {
    (*g_kernel)();
    g_fiber->done = true;
    _longjmp(g_scheduler, 1);
}
// Runs a fiber up to its next point.
__attribute__((noinline)) inline void run(Fiber& f) {
    g_fiber = &f;
    if (_setjmp(g_scheduler)) return;
    if (f.begun) _longjmp(f.go_on, 1);
    f.begun = true;
    setcontext(&f.begin);
}

// Runs `ctas` blocks of `threads` as one cluster, block `first` ahead; false where threads wait for
// others that never come.
inline bool run_blocks(int ctas, int threads, unsigned first, size_t dynamic,
                       const std::function<void()>& kernel) {
    constexpr size_t kStack = 96 << 10;
    Cluster cl;
    cl.ctas = std::vector<Cta>(ctas);
    cl.all.threads = ctas * threads;
    std::vector<Fiber> fibers(ctas * threads);
    static std::vector<std::unique_ptr<char[]>> stacks;
    while (stacks.size() < fibers.size()) stacks.emplace_back(new char[kStack]);
    g_kernel = &kernel;
    g_block = {first, 0, 0};
    for (int c = 0; c < ctas; ++c) {
        Cta& cta = cl.ctas[c];
        cta.space.reset(new char[dynamic + 64]);
        memset(cta.space.get(), 0xEE, dynamic + 64);
        cta.dynamic = cta.space.get() + (-(uintptr_t)cta.space.get() & 15);
        cta.all.threads = threads;
        cta.warps = std::vector<Warp>(threads / 32);
        for (auto& w : cta.warps) w.meet.threads = 32;
        cta.rank = c;
        cta.cluster = &cl;
        for (int t = 0; t < threads; ++t) {
            Fiber& f = fibers[c * threads + t];
            f.thread = {(unsigned)t, 0, 0};
            f.cta = &cta;
            getcontext(&f.begin);
            f.begin.uc_stack.ss_sp = stacks[c * threads + t].get();
            f.begin.uc_stack.ss_size = kStack;
            f.begin.uc_link = nullptr;
            makecontext(&f.begin, fiber_main, 0);
        }
    }
    for (size_t left = fibers.size(); left;) {
        uint64_t before = (uint64_t)cl.all.turn - left;      // every step makes it larger
        for (auto& c : cl.ctas) {
            before += c.all.turn;
            for (auto& w : c.warps) before += w.meet.turn;
        }
        for (auto& f : fibers) {
            if (f.done) continue;
            run(f);
            left -= f.done;
        }
        uint64_t after = (uint64_t)cl.all.turn - left;
        for (auto& c : cl.ctas) {
            after += c.all.turn;
            for (auto& w : c.warps) after += w.meet.turn;
        }
        if (left && after == before) return false;
    }
    return true;
}

// ---------------------------------------------------------- warps and blocks
template <class T> uint64_t bits_of(T x) {
    uint64_t u = 0;
    memcpy(&u, &x, sizeof x);
    return u;
}
template <class T> T from_bits(uint64_t u) {
    T x;
    memcpy(&x, &u, sizeof x);
    return x;
}
template <class F> uint64_t warp_op(uint64_t mine, F f) {
    Warp& w = g_fiber->cta->warps[threadIdx.x / 32];
    w.value[threadIdx.x & 31] = mine;
    reach(w.meet);
    const uint64_t r = f(w.value);
    reach(w.meet);
    return r;
}
template <class T> T __shfl_xor_sync(unsigned, T x, int o) {
    const int l = threadIdx.x & 31;
    return from_bits<T>(warp_op(bits_of(x), [&](uint64_t* v) { return v[l ^ o]; }));
}
template <class T> T __shfl_sync(unsigned, T x, int o) {
    return from_bits<T>(warp_op(bits_of(x), [&](uint64_t* v) { return v[o & 31]; }));
}
inline unsigned __ballot_sync(unsigned, bool p) {
    return (unsigned)warp_op(p, [&](uint64_t* v) {
        uint64_t r = 0;
        for (int i = 0; i < 32; ++i) r |= (v[i] ? uint64_t(1) : 0) << i;
        return r;
    });
}
inline uint32_t __reduce_max_sync(unsigned, uint32_t x) {
    return (uint32_t)warp_op(x, [](uint64_t* v) { return *std::max_element(v, v + 32); });
}
inline bool g_no_minimum;              // plants a reduction in which no lane takes part
inline uint32_t __reduce_min_sync(unsigned, uint32_t x) {
    const uint32_t r =
        (uint32_t)warp_op(x, [](uint64_t* v) { return *std::min_element(v, v + 32); });
    return g_no_minimum ? 0xffffffffu : r;
}
inline uint32_t __reduce_or_sync(unsigned, uint32_t x) {
    return (uint32_t)warp_op(x, [](uint64_t* v) {
        uint64_t r = 0;
        for (int i = 0; i < 32; ++i) r |= v[i];
        return r;
    });
}
inline void __syncwarp() { reach(g_fiber->cta->warps[threadIdx.x / 32].meet); }
inline void __syncthreads() { reach(g_fiber->cta->all); }
inline int __syncthreads_count(bool p) {
    Cta& c = *g_fiber->cta;
    c.count += p;
    __syncthreads();
    const int r = c.count;
    __syncthreads();
    if (threadIdx.x == 0) c.count = 0;
    __syncthreads();
    return r;
}
inline int atomicAdd(int* p, int x) {
    const int old = *p;
    *p += x;
    return old;
}
inline unsigned long long atomicOr(unsigned long long* p, unsigned long long x) {
    const unsigned long long old = *p;
    *p |= x;
    return old;
}
namespace cooperative_groups {
struct cluster_group {
    int block_rank() const { return g_fiber->cta->rank; }
    int num_blocks() const { return (int)g_fiber->cta->cluster->ctas.size(); }
    void barrier_arrive() const {}
    void barrier_wait() const { sync(); }
    void sync() const { reach(g_fiber->cta->cluster->all); }
    template <class T> T* map_shared_rank(T* p, int rank) const {
        const Cta* mine = g_fiber->cta;
        return reinterpret_cast<T*>(mine->cluster->ctas[rank].dynamic +
                                    ((char*)p - mine->dynamic));
    }
};
inline cluster_group this_cluster() { return {}; }
}  // namespace cooperative_groups
namespace cg = cooperative_groups;

// ------------------------------------------------------------- types, numbers
struct float2 { float x, y; };
struct alignas(16) float4 { float x, y, z, w; };
struct uint2 { uint32_t x, y; };
struct alignas(16) uint4 { uint32_t x, y, z, w; };
inline float2 make_float2(float a, float b) { return {a, b}; }
inline float4 make_float4(float a, float b, float c, float d) { return {a, b, c, d}; }
inline uint32_t __float_as_uint(float x) { return std::bit_cast<uint32_t>(x); }
inline float __uint_as_float(uint32_t x) { return std::bit_cast<float>(x); }
inline float __int_as_float(int x) { return std::bit_cast<float>(x); }
inline float __fmul_rn(float a, float b) { return a * b; }
inline float __fmaf_rn(float a, float b, float c) { return std::fma(a, b, c); }
inline float __log2f(float x) { return std::log2(x); }
inline int __ffs(unsigned x) { return __builtin_ffs((int)x); }
inline int __ffsll(long long x) { return __builtin_ffsll(x); }
inline int __popc(unsigned x) { return __builtin_popcount(x); }
inline int __popcll(unsigned long long x) { return __builtin_popcountll(x); }
template <class T> T __ldg(const T* p) { return *p; }

struct __half { _Float16 v; };
struct __half2 { __half x, y; };
struct __nv_bfloat16 { uint16_t v; };
struct __nv_bfloat162 { __nv_bfloat16 x, y; };
inline float to_f32(float x) { return x; }
inline float to_f32(__half x) { return (float)x.v; }
inline float to_f32(__nv_bfloat16 x) { return __uint_as_float((uint32_t)x.v << 16); }
template <class T> T from_f32(float x);
template <> inline float from_f32<float>(float x) { return x; }
template <> inline __half from_f32<__half>(float x) { return {(_Float16)x}; }
template <> inline __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {      // of -inf and the like
    return {(uint16_t)(__float_as_uint(x) >> 16)};
}
inline float2 __half22float2(__half2 h) { return {to_f32(h.x), to_f32(h.y)}; }
template <class T2> T2 __hmax2(T2 a, T2 b) {                              // NaN is passed over
    using T = decltype(a.x);
    return {from_f32<T>(fmaxf(to_f32(a.x), to_f32(b.x))),
            from_f32<T>(fmaxf(to_f32(a.y), to_f32(b.y)))};
}
template <class T2> float __low2float(T2 a) { return to_f32(a.x); }
template <class T2> float __high2float(T2 a) { return to_f32(a.y); }

// What rnnt_labels.cuh gives the kernels.
template <int UB> struct Unit;
template <> struct Unit<16> { using type = uint4; };
template <> struct Unit<8> { using type = uint2; };
template <> struct Unit<4> { using type = uint32_t; };
template <> struct Unit<2> { using type = uint16_t; };
template <typename T, int UB> union Pack {
    typename Unit<UB>::type raw;
    T e[UB / (int)sizeof(T)];
    Pack() {}
};
inline void wait_for_previous() {}
inline void let_next_start() {}
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

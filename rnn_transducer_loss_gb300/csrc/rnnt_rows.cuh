// rnnt_rows.cuh -- rows of V logits as the operators that learn from a teacher read them
// (rnnt_distill.cu, rnnt_sample.cu): 16-byte vectors of a row at any alignment, packed arithmetic,
// reductions of a warp and of a block.
#pragma once
#include <atomic>
#include <cmath>

#include "rnnt_labels.cuh"

namespace rnnt_rows {
using namespace rnnt_labels;

constexpr unsigned kAll = 0xffffffffu;
constexpr double kLog2e = 1.4426950408889634074;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger, NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Order-preserving integers; -0 counts as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Keys in the order of the values, the lower element first where they are equal.  Never 0.
__device__ __forceinline__ uint64_t key_of(float x, int element) {
    return (uint64_t)ordered(x) << 32 | (uint32_t)~element;
}
__device__ __forceinline__ float value_of(uint64_t key) { return unordered((uint32_t)(key >> 32)); }
__device__ __forceinline__ int element_of(uint64_t key) { return (int)~(uint32_t)key; }

template <typename V>
__device__ __forceinline__ V warp_sum(V x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {           // NaN is passed over
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Four sums at once: half of the values go with each half of the lanes, so 6 exchanges instead of 20.
__device__ __forceinline__ float4 warp_sum4(float a, float b, float c, float d) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, right = lane & 8;
    float x = (up ? c : a) + __shfl_xor_sync(kAll, up ? a : c, 16);
    float y = (up ? d : b) + __shfl_xor_sync(kAll, up ? b : d, 16);
    x = (right ? y : x) + __shfl_xor_sync(kAll, right ? x : y, 8);
    x += __shfl_xor_sync(kAll, x, 4);
    x += __shfl_xor_sync(kAll, x, 2);
    x += __shfl_xor_sync(kAll, x, 1);
    return make_float4(__shfl_sync(kAll, x, 0), __shfl_sync(kAll, x, 8), __shfl_sync(kAll, x, 16),
                       __shfl_sync(kAll, x, 24));
}
__device__ __forceinline__ float reciprocal(float x) {          // to one step
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rounded_reciprocal(float x) {  // of x >= 1: a Newton step more
    const float r = reciprocal(x);
    return __fmaf_rn(r, __fmaf_rn(-x, r, 1.0f), r);
}
__device__ __forceinline__ float warp_max_nan(float x) {
    float y;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
template <typename Key>
__device__ __forceinline__ Key warp_largest(Key x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Key y = __shfl_xor_sync(kAll, x, o);
        x = y > x ? y : x;
    }
    return x;
}

// Sorted in descending order over the warp (bitonic).
__device__ __forceinline__ float warp_sorted(float x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o; o >>= 1) {
            const float y = __shfl_xor_sync(kAll, x, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0 || size == 32);
            x = larger ? fmaxf(x, y) : fminf(x, y);
        }
    }
    return x;
}

// A row of V elements from x on, as the 16-byte units of memory it lies in: element e of vector j is
// x[j * E + e - off].  What of the first and the last unit is not the row's reads as -inf and
// is neither loaded nor stored.
// WHOLE: every row is made of whole units.
template <typename T, bool WHOLE = false>
struct Row {
    static constexpr int E = 16 / (int)sizeof(T);
    const T* x;
    int V, off, n;

    __device__ __forceinline__ Row(const T* row, int size) : x(row), V(size) {
        off = WHOLE ? 0 : (int)((uintptr_t)row & 15) / (int)sizeof(T);
        n = (off + V + E - 1) / E;
    }
    __device__ __forceinline__ bool whole(int j) const {
        return WHOLE || (j * E >= off && (j + 1) * E <= off + V);
    }
    __device__ __forceinline__ Pack<T, 16> load(int j) const {
        Pack<T, 16> v;
        if (whole(j)) {
            v.raw = reinterpret_cast<const uint4*>(x - off)[j];
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = j * E + e - off;
                v.e[e] = (unsigned)i < (unsigned)V ? x[i] : from_f32<T>(-INFINITY);
            }
        }
        return v;
    }
    // To a row at the same alignment.
    __device__ __forceinline__ void store(T* y, int j, const Pack<T, 16>& v) const {
        if (whole(j)) {
            reinterpret_cast<uint4*>(y - off)[j] = v.raw;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = j * E + e - off;
                if ((unsigned)i < (unsigned)V) y[i] = v.e[e];
            }
        }
    }
};

// ------------------------------------------------------ packed arithmetic
// Two float32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d)
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d)
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d)
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return reinterpret_cast<float2&>(d);
}
// The elements of a vector, two by two, and back (rounded to the type).
__device__ __forceinline__ void unpack(const Pack<float, 16>& v, float2 (&y)[2]) {
    y[0] = make_float2(v.e[0], v.e[1]);
    y[1] = make_float2(v.e[2], v.e[3]);
}
__device__ __forceinline__ void unpack(const Pack<__half, 16>& v, float2 (&y)[4]) {
    const __half2* h = reinterpret_cast<const __half2*>(&v.raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __half22float2(h[i]);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 16>& v, float2 (&y)[4]) {
    const uint32_t w[4] = {v.raw.x, v.raw.y, v.raw.z, v.raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void pack(Pack<float, 16>& v, const float2 (&y)[2]) {
    v.e[0] = y[0].x, v.e[1] = y[0].y, v.e[2] = y[1].x, v.e[3] = y[1].y;
}
__device__ __forceinline__ void pack(Pack<__half, 16>& v, const float2 (&y)[4]) {
    __half2* h = reinterpret_cast<__half2*>(&v.raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22half2_rn(y[i]);
}
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, 16>& v, const float2 (&y)[4]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v.raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(y[i]);
}
// The larger of two vectors' elements, and the largest element of one; NaN where there is one.
__device__ __forceinline__ Pack<float, 16> larger(const Pack<float, 16>& a, const Pack<float, 16>& b) {
    Pack<float, 16> m;
#pragma unroll
    for (int e = 0; e < 4; ++e) m.e[e] = max_nan(a.e[e], b.e[e]);
    return m;
}
template <typename T> struct Two;
template <> struct Two<__half> { using type = __half2; };
template <> struct Two<__nv_bfloat16> { using type = __nv_bfloat162; };
template <typename T>
__device__ __forceinline__ Pack<T, 16> larger(const Pack<T, 16>& a, const Pack<T, 16>& b) {
    using T2 = typename Two<T>::type;
    const T2 *x = reinterpret_cast<const T2*>(&a.raw), *y = reinterpret_cast<const T2*>(&b.raw);
    Pack<T, 16> m;
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<T2*>(&m.raw)[i] = __hmax2_nan(x[i], y[i]);
    return m;
}
// Of the first and of the second half of a vector's elements.
__device__ __forceinline__ float2 half_maxima(const Pack<float, 16>& m) {
    return make_float2(max_nan(m.e[0], m.e[1]), max_nan(m.e[2], m.e[3]));
}
template <typename T>
__device__ __forceinline__ float2 half_maxima(const Pack<T, 16>& m) {
    using T2 = typename Two<T>::type;
    const T2* h = reinterpret_cast<const T2*>(&m.raw);
    const T2 a = __hmax2_nan(h[0], h[1]), b = __hmax2_nan(h[2], h[3]);
    return make_float2(max_nan(__low2float(a), __high2float(a)),
                       max_nan(__low2float(b), __high2float(b)));
}
// The elements of a vector that are at least `least`, or above it, as bits.
template <bool STRICT = false>
__device__ __forceinline__ uint32_t reaching(const Pack<float, 16>& v, float least) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m |= (STRICT ? v.e[e] > least : v.e[e] >= least) ? 1u << e : 0u;
    return m;
}
template <bool STRICT = false, typename T>
__device__ __forceinline__ uint32_t reaching(const Pack<T, 16>& v, T least) {
    using T2 = typename Two<T>::type;
    T2 two;
    two.x = least, two.y = least;
    const T2* h = reinterpret_cast<const T2*>(&v.raw);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m |= (STRICT ? __hgt2_mask(h[i], two) : __hge2_mask(h[i], two)) & (0x00020001u << (2 * i));
    return (m | m >> 16) & 0xffu;
}
// The least value of the type that is not below x, and the lowest finite one.
template <typename T> __device__ __forceinline__ T not_below(float x);
template <> __device__ __forceinline__ float not_below<float>(float x) { return x; }
template <> __device__ __forceinline__ __half not_below<__half>(float x) {
    return __float2half_ru(x);
}
template <> __device__ __forceinline__ __nv_bfloat16 not_below<__nv_bfloat16>(float x) {
    return __float2bfloat16_ru(x);
}
template <typename T>
__device__ constexpr float lowest() {
    return sizeof(T) == 4 ? -3.40282347e38f : std::is_same_v<T, __half> ? -65504.0f : -3.38953139e38f;
}

template <typename T>
__device__ __forceinline__ Pack<T, 16> all_minus_inf() {
    Pack<T, 16> v;
#pragma unroll
    for (int e = 0; e < 16 / (int)sizeof(T); ++e) v.e[e] = from_f32<T>(-INFINITY);
    return v;
}

// 2^((y - ref) c), c in two parts: rounded to one float32 it would shift all of a row's terms by up
// to 6e-8 of their exponent the same way, and with them the sum's logarithm.  Both parts are above 0,
// so that y = -inf gives 0.
inline void parts_below(double c, float& hi, float& lo) {
    hi = (float)c;
    if ((double)hi >= c) hi = std::nextafter(hi, 0.0f);
    lo = (float)(c - (double)hi);
}
// ex2.approx comes out low on average: over all float32 of a binary order by 2.2e-8 for exponents above
// -1 and by 4.9e-8 to 5.2e-8 in every order below.  kLow, in the exponent, makes up for 2.2e-8: logarithms
// of sums are then off by -2e-8 (exponents below -1) to 3e-8 (all above -1) on average, logf included.
constexpr float kLow = 3.2e-8f;
struct Exponent {
    float2 ref, hi, lo;                    // -ref, c
    __device__ __forceinline__ Exponent(float at, float h, float l)
        : ref(make_float2(-at, -at)), hi(make_float2(h, h)), lo(make_float2(l, l)) {}
    __device__ __forceinline__ float2 operator()(float2 y) const {
        const float2 d = add2(y, ref), t = fma2(d, hi, fma2(d, lo, make_float2(kLow, kLow)));
        return make_float2(ex2(t.x), ex2(t.y));
    }
    __device__ __forceinline__ float operator()(float y) const {
        const float d = y + ref.x;
        return ex2(__fmaf_rn(d, hi.x, __fmaf_rn(d, lo.x, kLow)));
    }
};
// The terms of a vector and their sum, as a tree.
template <typename T, int H>
__device__ __forceinline__ float terms_of(const Pack<T, 16>& v, const Exponent& f, float2 (&e)[H]) {
    unpack(v, e);
#pragma unroll
    for (int i = 0; i < H; ++i) e[i] = f(e[i]);
    if constexpr (H == 4) {
        const float2 s = add2(add2(e[0], e[1]), add2(e[2], e[3]));
        return s.x + s.y;
    } else {
        const float2 s = add2(e[0], e[1]);
        return s.x + s.y;
    }
}

// ------------------------------------------------------------ groups of threads
// A row is taken by a group: a warp, or a whole block of G threads.
template <int G>
struct Group {
    static constexpr int WARPS = G / 32;
    struct Space { float f[2 * WARPS]; };  // of a block; a warp needs none
    __device__ static __forceinline__ int rank() { return G == 32 ? threadIdx.x & 31 : threadIdx.x; }
    __device__ static __forceinline__ void sync() {
        if constexpr (G == 32) __syncwarp();
        else __syncthreads();
    }
    __device__ static __forceinline__ float max(float x, Space& s) {
        x = warp_max_nan(x);
        if constexpr (G > 32) {
            if ((threadIdx.x & 31) == 0) s.f[threadIdx.x >> 5] = x;
            __syncthreads();
            x = s.f[0];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) x = max_nan(x, s.f[w]);
        }
        return x;
    }
    // Needs a barrier between two of one kind.
    __device__ static __forceinline__ float sum(float x, Space& s) {
        x = warp_sum(x);
        if constexpr (G > 32) {
            if ((threadIdx.x & 31) == 0) s.f[WARPS + (threadIdx.x >> 5)] = x;
            __syncthreads();
            x = s.f[WARPS];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) x += s.f[WARPS + w];
        }
        return x;
    }
};

// ------------------------------------------------ rows through shared memory
// Every group has a ring of stages; a row comes by one bulk copy of the whole units it lies in,
// announced at the stage's mbarrier, and is laid out in the stage as in memory.  Units that
// reach past the tensor's ends are not copied: their elements are loaded one by one.
constexpr int kWaitPolls = 1 << 22;        // then a wait gives up

__device__ __forceinline__ uint32_t shared_at(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint64_t* bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_at(bar)) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void fence_proxy_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_at(bar)),
                 "r"(bytes) : "memory");
    if (bytes)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
            ::"r"(shared_at(dst)), "l"(src), "r"(bytes), "r"(shared_at(bar)) : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(shared_at(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// A wait that gives up reports it, and later ones of the thread poll once: the kernel ends soon.
__device__ __forceinline__ void mbar_wait(uint64_t* bar, uint32_t parity, int& polls,
                                          int32_t* status) {
    for (int i = 0; i < polls; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred q;\n mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n"
            " selp.b32 %0, 1, 0, q;\n}"
            : "=r"(ok) : "r"(shared_at(bar)), "r"(parity) : "memory");
        if (ok) return;
    }
    polls = 1;
    if (status) *status = RNNT_TIMEOUT;
}

// A row in a stage: vectors as Row has them.
template <typename T, int G, bool WHOLE = false>
struct Staged {
    static constexpr int E = 16 / (int)sizeof(T);
    Row<T, WHOLE> r;
    uint4* s;
    int lo, hi;                            // the vectors that the copy brings

    // begin, end: of the tensor.  Rows shorter than a unit share its first and last one.
    __device__ __forceinline__ Staged(const T* x, int V, uint4* stage, const T* begin, const T* end)
        : r(x, V), s(stage) {
        const uintptr_t at = (uintptr_t)x - r.off * sizeof(T);
        lo = !WHOLE && at < (uintptr_t)begin ? 1 : 0;
        hi = !WHOLE && at + (uintptr_t)r.n * 16 > (uintptr_t)end ? r.n - 1 : r.n;
    }
    __device__ __forceinline__ void fetch(uint64_t* bar) const {       // by one thread
        const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16u : 0u;
        bulk_load(s + lo, reinterpret_cast<const uint4*>(r.x - r.off) + lo, bytes, bar);
    }
    // After the copy has arrived: what it did not bring, and -inf in place of what is not the row's.
    __device__ __forceinline__ void complete() const {
        if (WHOLE || (r.off == 0 && r.V % E == 0)) return;
        const int i = Group<G>::rank();
        T* e = reinterpret_cast<T*>(s);
        if (i < 2 * E) {
            const int at = i < E ? i : (r.n - 1) * E + i - E, el = at - r.off;
            if (i < E || r.n > 1) {
                if ((unsigned)el >= (unsigned)r.V) e[at] = from_f32<T>(-INFINITY);
                else if (i < E ? lo > 0 || hi <= lo : hi < r.n) e[at] = r.x[el];
            }
        }
        Group<G>::sync();
    }
    __device__ __forceinline__ Pack<T, 16> at(int j) const {
        Pack<T, 16> v;
        v.raw = s[j];
        return v;
    }
    __device__ __forceinline__ T& element(int i) const { return reinterpret_cast<T*>(s)[r.off + i]; }
};

// Device-side memory limits of kernels, raised once per device by `raise()`.
template <typename F>
inline bool prepared_once(std::atomic<bool>* done, F&& raise) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    if (done[dev].load(std::memory_order_acquire)) return true;
    const bool ok = raise();
    if (ok) done[dev].store(true, std::memory_order_release);
    else cudaGetLastError();
    return ok;
}

}  // namespace rnnt_rows

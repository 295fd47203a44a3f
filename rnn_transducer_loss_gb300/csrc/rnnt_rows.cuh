// rnnt_rows.cuh -- rows of V logits as the operators that learn from a teacher read them
// (rnnt_distill.cu, rnnt_sample.cu): 16-byte vectors of a row at any alignment, packed arithmetic,
// reductions of a warp and of a block.
#pragma once
#include <atomic>

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
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
    return x;
}
__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = max_nan(x, __shfl_xor_sync(kAll, x, o));
    return x;
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

// A row of V elements from x on, as the 16-byte units of memory it lies in: element e of vector j is
// x[j * E + e - off].  What of the first and the last unit is not the row's reads as -inf and
// is neither loaded nor stored.
template <typename T>
struct Row {
    static constexpr int E = 16 / (int)sizeof(T);
    const T* x;
    int V, off, n;

    __device__ __forceinline__ Row(const T* row, int size) : x(row), V(size) {
        off = (int)((uintptr_t)row & 15) / (int)sizeof(T);
        n = (off + V + E - 1) / E;
    }
    __device__ __forceinline__ bool whole(int j) const {
        return j * E >= off && (j + 1) * E <= off + V;
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

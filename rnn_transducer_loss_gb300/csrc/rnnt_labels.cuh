// rnnt_labels.cuh -- what the label-side operators (rnnt_embed.cu, rnnt_beam.cu) share:
// element types, wide memory units, small host helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "rnnt_gb300.h"

namespace rnnt_labels {

// Storage types; every sum, product and statistic is float32 or wider.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// A memory unit of UB bytes: the widest access that every address and stride
// of a call allows (16 bytes where all are multiples of 16).
template <int UB> struct Unit;
template <> struct Unit<16> { using type = uint4; };
template <> struct Unit<8> { using type = uint2; };
template <> struct Unit<4> { using type = uint32_t; };
template <> struct Unit<2> { using type = uint16_t; };
template <> struct Unit<1> { using type = uint8_t; };

// The elements of one unit.
template <typename T, int UB>
union Pack {
    typename Unit<UB>::type raw;
    T e[UB / (int)sizeof(T)];
    __device__ Pack() {}
};

// A kernel launched by launch_after may start while the kernel before it in the stream runs its
// last blocks; all its blocks call wait_for_previous, before they touch what that kernel writes.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Params, typename... Args>
inline bool launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t shared,
                         cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool valid_dtype(int dt) { return dt == RNNT_F32 || dt == RNNT_F16 || dt == RNNT_BF16; }
inline int elem_size(int dt) { return dt == RNNT_F32 ? 4 : 2; }

// Largest of 16, 8, 4, 2, 1 that divides every bit pattern or-ed into x.
inline int unit_of(uint64_t x) {
    const uint64_t low = (x | 16) & (~(x | 16) + 1);
    return (int)low;
}

inline bool overlaps(const void* a, uint64_t an, const void* b, uint64_t bn) {
    const uint64_t x = (uint64_t)(uintptr_t)a, y = (uint64_t)(uintptr_t)b;
    return x < y + bn && y < x + an;
}

// Calls f(T{}) with the storage type of dt.
template <typename F>
inline auto with_type(int dt, F&& f) {
    if (dt == RNNT_F32) return f(float{});
    if (dt == RNNT_F16) return f(__half{});
    return f(__nv_bfloat16{});
}

// Sets *status (if there is one) to RNNT_OK ahead of a call's kernels.
inline bool clear_status(int32_t* status, cudaStream_t st) {
    return !status || cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess;
}

inline rnnt_status_t launched() {
    return cudaGetLastError() == cudaSuccess ? RNNT_OK : RNNT_LAUNCH_FAILED;
}

}  // namespace rnnt_labels

// rowvec.cuh - rows of fp32, bf16 or fp16 elements as fp32 values: 16-byte
// vectors where every row starts on a 16-byte boundary, single elements
// otherwise.  Used by the row-wise operators (embedding.cu, rms_norm.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "carbon_internal.h"

namespace carbon {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(int8_t v) { return (float)v; }

// One rounding, to nearest-even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements of T.  N = 16 / sizeof(T) (one 16-byte access, the
// address 16-byte aligned) or 1.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T e[N];
};

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// By value: one access where v is in memory.
template <typename T, int N>
__device__ __forceinline__ void widen(const Pack<T, N> v, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(v.e[i]);
}

template <typename T, int N>
__device__ __forceinline__ void load_f32(const T *p, float (&f)[N]) {
    widen(*reinterpret_cast<const Pack<T, N> *>(p), f);
}

template <typename T, int N>
__device__ __forceinline__ void store_f32(T *p, const float (&f)[N]) {
    Pack<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.e[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Pack<T, N> *>(p) = v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// Whether every pointer (null ones too) is a multiple of `size`, a power of two.
template <typename... P>
inline bool aligned_to(size_t size, const P *...p) {
    return (((0 | ... | reinterpret_cast<uintptr_t>(p)) & (size - 1)) == 0);
}
inline bool aligned16(const void *p) { return aligned_to(16, p); }

inline size_t dtype_size(int dtype) { return dtype == CARBON_F32 ? 4 : 2; }

}  // namespace carbon

// Conversions between element types and binary32, and 16-byte vectors of elements, for
// the operators' kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "params.h"

namespace gb300 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements moved at once: N * sizeof(T) is 16, 32, or the size of one element.
template <typename T, int N>
struct alignas(N * sizeof(T) >= 16 ? 16 : sizeof(T)) Pack {
  T v[N];
};

// A plain (coherent) load: the operators may run in place.
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&f)[N]) {
  const Pack<T, N> x = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = to_f32(x.v[i]);
}

template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&f)[N]) {
  Pack<T, N> x;
#pragma unroll
  for (int i = 0; i < N; ++i) x.v[i] = from_f32<T>(f[i]);
  *reinterpret_cast<Pack<T, N>*>(p) = x;
}

// An index in device memory was out of its range: recorded once, not followed.
__device__ __forceinline__ void record_bad_index(uint32_t* status, uint32_t site) {
  atomicCAS(status, 0u, (kDevBadIndex << 24) | (site << 16) | (blockIdx.x & 0xFFFFu));
}

}  // namespace gb300

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

// N elements moved at once: N * sizeof(T) is 16, 32, or the size of one element.  Kept as
// loaded until unpack, pairs of 16-bit elements in a register.
template <typename T, int N>
struct alignas(N * sizeof(T) >= 16 ? 16 : sizeof(T)) Pack {
  T v[N];
};

__device__ __forceinline__ float2 pair_f32(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ float2 pair_f32(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ void pair_rn(__half2& d, float a, float b) { d = __floats2half2_rn(a, b); }
__device__ __forceinline__ void pair_rn(__nv_bfloat162& d, float a, float b) {
  d = __floats2bfloat162_rn(a, b);
}
template <typename T> struct PairOf { using type = __half2; };
template <> struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };

template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<T, N>& x, float (&f)[N]) {
  if constexpr (sizeof(T) == 4 || N % 2 != 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(x.v[i]);
  } else {
    using P = typename PairOf<T>::type;
    const P* w = reinterpret_cast<const P*>(&x);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 p = pair_f32(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> pack(const float (&f)[N]) {
  Pack<T, N> x;
  if constexpr (sizeof(T) == 4 || N % 2 != 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) x.v[i] = from_f32<T>(f[i]);
  } else {
    using P = typename PairOf<T>::type;
    P* w = reinterpret_cast<P*>(&x);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) pair_rn(w[i], f[2 * i], f[2 * i + 1]);
  }
  return x;
}

// A plain (coherent) load: the operators may run in place.
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&f)[N]) {
  unpack(*reinterpret_cast<const Pack<T, N>*>(p), f);
}

template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&f)[N]) {
  *reinterpret_cast<Pack<T, N>*>(p) = pack<T, N>(f);
}

// v as the sum of P parts, each the nearest value to what the parts before it leave (zero
// after an infinity).
template <typename T, int P>
__device__ __forceinline__ void split_f32(float v, T (&part)[P]) {
#pragma unroll
  for (int j = 0; j < P; ++j) {
    part[j] = from_f32<T>(v);
    const float f = to_f32(part[j]);
    v = isinf(f) ? 0.0f : v - f;
  }
}

// A row of Up times u, in binary32: what the matrix instructions' sum over the parts of u
// stands for, except that they make a NaN of an infinity in Up, times parts that are zero or of
// both signs.
template <typename T>
__device__ __forceinline__ float up_times_u(const T* up, const float* u, int32_t rank) {
  float sum = 0.0f;
  for (int32_t r = 0; r < rank; r += 8) {
    float w[8];
    unpack(*reinterpret_cast<const Pack<T, 8>*>(up + r), w);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(u[r + k], w[k], sum);
  }
  return sum;
}

// An index in device memory was out of its range: recorded once, not followed.
__device__ __forceinline__ void record_bad_index(uint32_t* status, uint32_t site) {
  atomicCAS(status, 0u, (kDevBadIndex << 24) | (site << 16) | (blockIdx.x & 0xFFFFu));
}

}  // namespace gb300

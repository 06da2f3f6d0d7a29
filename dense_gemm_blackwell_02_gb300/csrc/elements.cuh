// Conversions between element types and binary32, and 16-byte vectors of elements, for
// the operators' kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

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

// A row of u while its values are looked through, as the bit patterns of magnitudes: the
// largest that is not an infinity (a NaN's is above all of them), and the smallest, less one,
// so that zeros wrap round and do not count.
struct RowRange {
  static constexpr uint32_t kInf = 0x7f800000u;
  uint32_t most = 0, least = 0xFFFFFFFFu;
  __device__ __forceinline__ void add(float x) {
    const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
    most = max(most, m == kInf ? 0u : m);
    least = min(least, m - 1u);
  }
  // Of the `lanes` neighbouring threads that share the row.
  __device__ __forceinline__ void join(int lanes) {
    for (int off = lanes / 2; off > 0; off >>= 1) {
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, off));
      least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, off));
    }
  }
};

// How a row of u goes into its 16-bit parts.  A value times `inv` is split; the sum over the
// parts times `scale`, the inverse, is the row's term.  scale is NaN for a row with a NaN, and
// negative for a row whose parts do not hold every value, to be multiplied in binary32.
//
// bf16 has binary32's range, short of the parts of values below 2^-100 (and of what rounds up
// to an infinity).
// fp16: the largest value comes to 2^14..2^15, and parts end at 2^-24, so that they leave up to
// 2^-25 of a value.  What is then below `least`, 2^-5 (2^-20 of the largest at most), would lose
// more than 2^-20 of itself in a binary32 result, and below 2^-8 more than 2^-17 in a 16-bit one.
// Such values go into a second window: 2^(10 - log2 least) times themselves, below 2^15 again,
// a sum of its own times `scale_low` (0: none of the row's values are there).  Two windows reach
// 2^-39 (16-bit results: 2^-45) of the row's largest.  Of 64 normally distributed values one is in
// the second window in one row of 5000 (40000), but a nearly dead rank has one in every row.
struct RowFactor {
  float inv = 1.0f, scale = 1.0f, least = 0.0f, inv_low = 0.0f, scale_low = 0.0f;
  // A value of u in either window.
  __device__ __forceinline__ float high(float u) const {
    const float x = u * inv;
    return fabsf(x) < least ? 0.0f : x;
  }
  __device__ __forceinline__ float low(float u) const {
    return fabsf(u * inv) < least ? u * inv_low : 0.0f;
  }
};
__host__ __device__ constexpr float window_least(bool f32_out) { return f32_out ? 0x1p-5f : 0x1p-8f; }
__host__ __device__ constexpr float window_step(bool f32_out) { return 0x1p15f / window_least(f32_out); }
template <typename T>
__device__ __forceinline__ RowFactor row_factor(const RowRange& r, bool f32_out) {
  RowFactor f;
  uint32_t lowest = __float_as_uint(0x1p-100f);  // what is smaller is too small
  if constexpr (std::is_same<T, __half>::value) {
    const int32_t e = min(max((int32_t)(r.most >> 23), 15), 254);
    f.inv = __uint_as_float((uint32_t)(268 - e) << 23);
    f.scale = __uint_as_float((uint32_t)(e - 14) << 23);
    f.least = window_least(f32_out);
    const float first = f.least * f.scale, second = first / window_step(f32_out);
    if (r.least < __float_as_uint(first) - 1u) {
      f.inv_low = f.inv * window_step(f32_out);
      f.scale_low = f.scale / window_step(f32_out);
    }
    lowest = max(__float_as_uint(second), 1u);
    // (binary32 itself ends before the second window does)
    if (isinf(f.inv_low) || (f.inv_low != 0.0f && f.scale_low < 0x1p-126f)) lowest = __float_as_uint(first);
  }
  if (r.least < lowest - 1u || r.most > __float_as_uint(0x1.fep127f)) f.scale = -1.0f, f.scale_low = 0.0f;
  if (r.most > RowRange::kInf) f.scale = __int_as_float(0x7fc00000), f.scale_low = 0.0f;
  return f;
}

// A row of Up times u, in binary32: what the matrix instructions' sum over the parts of u
// stands for, except that they make a NaN of an infinity in Up, times parts that are zero or of
// both signs, and an infinity of a product next to binary32's end, and that fp16 parts lose what
// is far below the row's largest value.
template <typename T>
__device__ __forceinline__ float up_times_u(const T* up, const float* u, int32_t rank) {
  float sum = 0.0f;
#pragma unroll 4
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

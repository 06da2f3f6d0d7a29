// Rotary positions with several axes: pair i of every head of token t turns by the angle
// theta = theta_i(positions[axis(i)][t]), whose cosine and sine come from tables:
//     a' = a cos - b sin,  b' = b cos + a sin          (the inverse negates sin)
// in binary32, rounded once to the element type.
//
// Six operations per pair against 4 elements moved: bound by HBM, so the kernel is one
// pass of 16-byte accesses.  A thread owns one vector of pairs of a head (two vectors of
// the head when a pair's halves lie apart, one when they are neighbours), reads its
// cosines and sines once, and turns that vector in `head_run` consecutive heads of the
// token, whose loads are all issued before the first use.
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRun = 4;  // heads whose loads are in flight together

// Whether one axis turns N pairs, whose bytes start at a multiple of N.
template <int N>
__device__ __forceinline__ bool one_axis(const uint8_t* axis) {
  if constexpr (N == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(axis);
    return w.x == w.y && w.x == (w.x & 0xFFu) * 0x01010101u;
  } else if constexpr (N == 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(axis);
    return w == (w & 0xFFu) * 0x01010101u;
  } else {
    return N == 2 ? axis[0] == axis[1] : true;
  }
}

// N values of a table's row (16-byte aligned for N >= 4, 8-byte for 2).
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&f)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + j));
      f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    f[0] = v.x, f[1] = v.y;
  } else {
    f[0] = __ldg(p);
  }
}

// NEIGH: neighbouring pairs.  V: elements per vector (1: no alignment is assumed).
template <typename T, bool NEIGH, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  // pairs per item: V with the halves apart (two vectors), V / 2 as neighbours (one; with
  // V = 1 two single elements)
  constexpr int kPairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  constexpr int kSpan = NEIGH ? 2 * kPairs : V;  // elements of one access
  grid_dependency_wait();
  grid_launch_dependents();

  const int lanes = min(p.items, kThreads);        // threads per (token, run of heads)
  const int groups = kThreads / lanes;             // ... of which a CTA holds this many
  const int g = (int)threadIdx.x / lanes;
  if (g >= groups) return;
  const int64_t q = (int64_t)blockIdx.x * groups + g;
  const int32_t t = (int32_t)(q / p.head_runs);
  if (t >= p.tokens) return;
  const int32_t h0 = (int32_t)(q - (int64_t)t * p.head_runs) * p.head_run;
  const int32_t nh = min(p.head_run, p.heads - h0);
  const T* x = static_cast<const T*>(p.x) + (int64_t)t * p.x_token + (int64_t)h0 * p.x_head;
  T* y = static_cast<T*>(p.y) + (int64_t)t * p.y_token + (int64_t)h0 * p.y_head;
  const int pair_items = (p.half + kPairs - 1) / kPairs;  // (exact unless V is 1)

  for (int item = (int)threadIdx.x - g * lanes; item < p.items; item += lanes) {
    if (item >= pair_items) {
      // past the pairs: copied, unless the operator runs in place
      if (static_cast<const void*>(p.x) == p.y) continue;
      const int d = 2 * p.half + (item - pair_items) * V;
      for (int k = 0; k < nh; ++k)
        *reinterpret_cast<Pack<T, V>*>(y + k * p.y_head + d) =
            *reinterpret_cast<const Pack<T, V>*>(x + k * p.x_head + d);
      continue;
    }
    const int i0 = item * kPairs;
    const int d0 = NEIGH ? 2 * i0 : i0, d1 = i0 + p.half;  // (d1: second halves)
    float a[kMaxRun][kSpan], b[kMaxRun][NEIGH ? 1 : kSpan];
#pragma unroll
    for (int k = 0; k < kMaxRun; ++k) {
      if (k >= nh) break;
      if constexpr (NEIGH && V == 1) {
        a[k][0] = to_f32(x[k * p.x_head + d0]);
        a[k][1] = to_f32(x[k * p.x_head + d0 + 1]);
      } else {
        load_f32<T, kSpan>(x + k * p.x_head + d0, a[k]);
        if constexpr (!NEIGH) load_f32<T, kSpan>(x + k * p.x_head + d1, b[k]);
      }
    }
    float c[kPairs], s[kPairs];
    if (V > 1 && one_axis<kPairs>(p.pair_axis + i0)) {
      // one position for the whole vector: its cosines and sines stand in a row
      const int64_t pos = p.positions[(int64_t)p.pair_axis[i0] * p.tokens + t];
      if (pos >= 0 && pos < p.num_positions) {
        load_row<kPairs>(p.cos + pos * p.half + i0, c);
        load_row<kPairs>(p.sin + pos * p.half + i0, s);
      } else {
        record_bad_index(p.status, kSitePosition);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) c[j] = 1.0f, s[j] = 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const int64_t pos = p.positions[(int64_t)p.pair_axis[i0 + j] * p.tokens + t];
        c[j] = 1.0f;
        s[j] = 0.0f;
        if (pos >= 0 && pos < p.num_positions) {
          c[j] = __ldg(p.cos + pos * p.half + i0 + j);
          s[j] = __ldg(p.sin + pos * p.half + i0 + j);
        } else {
          record_bad_index(p.status, kSitePosition);
        }
      }
    }
    if (p.inverse) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) s[j] = -s[j];
    }
#pragma unroll
    for (int k = 0; k < kMaxRun; ++k) {
      if (k >= nh) break;
      if constexpr (NEIGH) {
        float r[kSpan];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          r[2 * j] = a[k][2 * j] * c[j] - a[k][2 * j + 1] * s[j];
          r[2 * j + 1] = a[k][2 * j + 1] * c[j] + a[k][2 * j] * s[j];
        }
        if constexpr (V == 1) {
          y[k * p.y_head + d0] = from_f32<T>(r[0]);
          y[k * p.y_head + d0 + 1] = from_f32<T>(r[1]);
        } else {
          store_f32<T, kSpan>(y + k * p.y_head + d0, r);
        }
      } else {
        float ra[kSpan], rb[kSpan];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          ra[j] = a[k][j] * c[j] - b[k][j] * s[j];
          rb[j] = b[k][j] * c[j] + a[k][j] * s[j];
        }
        store_f32<T, kSpan>(y + k * p.y_head + d0, ra);
        store_f32<T, kSpan>(y + k * p.y_head + d1, rb);
      }
    }
  }
}

template <typename T, bool NEIGH, int V>
cudaError_t launch(RotaryParams& p, int sms, cudaStream_t stream) {
  const int pairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  p.items = p.half / pairs + (p.dim - 2 * p.half) / V;
  const int groups = kThreads / std::min(p.items, kThreads);
  // As many heads per thread as keep every SM busy with four CTAs; fewer tokens than that
  // spread their heads over more threads.
  p.head_run = 1;
  for (int run = kMaxRun; run > 1; run /= 2)
    if ((int64_t)p.tokens * ((p.heads + run - 1) / run) >= (int64_t)4 * sms * groups) {
      p.head_run = run;
      break;
    }
  p.head_runs = (p.heads + p.head_run - 1) / p.head_run;
  p.head_run = (p.heads + p.head_runs - 1) / p.head_runs;  // even runs
  const int64_t blocks = ((int64_t)p.tokens * p.head_runs + groups - 1) / groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<T, NEIGH, V>, p);
}

template <typename T>
cudaError_t by_layout(RotaryParams& p, bool neighbours, bool vec, int sms, cudaStream_t stream) {
  constexpr int V = 16 / (int)sizeof(T);
  if (neighbours)
    return vec ? launch<T, true, V>(p, sms, stream) : launch<T, true, 1>(p, sms, stream);
  return vec ? launch<T, false, V>(p, sms, stream) : launch<T, false, 1>(p, sms, stream);
}

}  // namespace

int rotary_vector(int elem) { return elem == kElemF32 ? 4 : 8; }

cudaError_t launch_rotary(RotaryParams p, int elem, bool neighbours, bool vec, int sms,
                          cudaStream_t stream) {
  switch (elem) {
    case kElemF16: return by_layout<__half>(p, neighbours, vec, sms, stream);
    case kElemBF16: return by_layout<__nv_bfloat16>(p, neighbours, vec, sms, stream);
    case kElemF32: return by_layout<float>(p, neighbours, vec, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gb300

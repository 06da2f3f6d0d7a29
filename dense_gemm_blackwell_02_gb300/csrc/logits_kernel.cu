// Logits before sampling: for every row i and token v
//     z = logits[i][v];  in the history: z = z > 0 ? z / rep : z * rep
//     c times generated: z -= freq * c + (c > 0 ? pres : 0);  z += biases of v
//     masked out: z = -inf
// in binary32, rounded once.
//
// A handful of operations per element: bound by HBM, one read and one write of the logits.
// A CTA owns one slice of one row's vocabulary.  It counts the row's whole history into a
// table in shared memory, one word per token of its slice (the history is short next to
// the vocabulary and comes from L2 after the row's first slice), then streams its logits
// past the table once.  Integer counts: the result does not depend on the atomics' order.
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 512;
constexpr int kVec = 8;            // logits per thread and step
constexpr int kTokens = 8;         // history tokens per thread in flight
constexpr int kMaxSlice = 16384;   // words of table: 64 KiB, three CTAs per SM
constexpr int kMinSlice = 2048;

// The table's word of a token: how often it was generated, and two flags.
constexpr uint32_t kInPrompt = 1u << 31;
constexpr uint32_t kHasBias = 1u << 30;
constexpr uint32_t kCount = kHasBias - 1u;

struct RowRules {
  float rep, freq, pres;
  int64_t bias0, bias1;
};

// One logit through the penalties and biases its word calls for.
__device__ __forceinline__ float adjust(float z, uint32_t word, int32_t v, const RowRules& r,
                                        const LogitsParams& p) {
  if (word & ~kHasBias) {
    z = z > 0.0f ? __fdiv_rn(z, r.rep) : z * r.rep;
    const uint32_t c = word & kCount;
    if (c) z = z - r.freq * (float)c - r.pres;
  }
  if (word & kHasBias) {
    int64_t lo = r.bias0, hi = r.bias1;  // the first entry not below v
    while (lo < hi) {
      const int64_t mid = lo + (hi - lo) / 2;
      if (p.bias_tokens[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    float w = 0.0f;
    for (; lo < r.bias1 && p.bias_tokens[lo] == v; ++lo) w += p.bias_values[lo];
    z += w;
  }
  return z;
}

// TABLE: there are histories or biases to look up.
template <typename TI, typename TO, bool TABLE>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ __align__(16) uint32_t table[];
  grid_dependency_wait();
  grid_launch_dependents();

  const int32_t row = (int32_t)(blockIdx.x / (uint32_t)p.slices);
  const int32_t part = (int32_t)(blockIdx.x - (uint32_t)row * (uint32_t)p.slices);
  const TI* in = static_cast<const TI*>(p.in) + (int64_t)row * p.in_stride;
  TO* out = static_cast<TO*>(p.out) + (int64_t)row * p.out_stride;
  // Rows of any alignment: positions are counted from the 16-byte boundary of the vectors
  // below the row's start, w = v + shift, so that vectors of kVec positions are aligned
  // (in input and output alike, else single elements are moved).
  const int32_t shift = (int32_t)((reinterpret_cast<uintptr_t>(in) / sizeof(TI)) % kVec);
  const bool vec = (int32_t)((reinterpret_cast<uintptr_t>(out) / sizeof(TO)) % kVec) == shift;
  const int32_t w0 = part * p.slice, w1 = min(w0 + p.slice, p.vocab + shift);
  if (w0 >= w1) return;  // (the last slice of a row with a small shift)

  RowRules r{1.0f, 0.0f, 0.0f, 0, 0};
  if constexpr (TABLE) {
    uint4* t4 = reinterpret_cast<uint4*>(table);
    for (int32_t i = (int32_t)threadIdx.x; i < p.slice / 4; i += kThreads) t4[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (p.tokens) {
      if (p.repetition) r.rep = p.repetition[row];
      if (p.frequency) r.freq = p.frequency[row];
      if (p.presence) r.pres = p.presence[row];
      const int64_t t0 = p.token_start[row], t1 = p.token_start[row + 1];
      const int64_t said = t0 + (p.prompt_len ? p.prompt_len[row] : 0);
      for (int64_t i0 = t0; i0 < t1; i0 += kThreads * kTokens) {
        int32_t v[kTokens];
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
          const int64_t i = i0 + j * kThreads + threadIdx.x;
          v[j] = i < t1 ? __ldg(p.tokens + i) : -1;
        }
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
          const int32_t w = v[j] + shift - w0;
          if (v[j] < 0 || v[j] >= p.vocab || w < 0 || w >= p.slice) continue;  // padding, or another slice's
          if (i0 + j * kThreads + threadIdx.x >= said) atomicAdd(table + w, 1u);
          else atomicOr(table + w, kInPrompt);
        }
      }
    }
    if (p.bias_tokens) {
      r.bias0 = p.bias_start[row];
      r.bias1 = p.bias_start[row + 1];
      for (int64_t i = r.bias0 + threadIdx.x; i < r.bias1; i += kThreads) {
        const int32_t v = p.bias_tokens[i];
        if (v < 0 || v >= p.vocab) continue;
        const int32_t w = v + shift - w0;
        if (w >= 0 && w < p.slice) atomicOr(table + w, kHasBias);
      }
    }
    __syncthreads();
  }

  const uint32_t* mask = nullptr;
  if (p.mask) {
    const int64_t m = p.mask_row ? p.mask_row[row] : row;
    if (m >= p.mask_count) {
      if (threadIdx.x == 0) record_bad_index(p.status, kSiteMaskRow);
    } else if (m >= 0) {
      mask = p.mask + m * p.mask_stride;
    }
  }

  for (int32_t w = w0 + (int32_t)threadIdx.x * kVec; w < w1; w += kThreads * kVec) {
    const int32_t v = w - shift;  // the first of kVec tokens; below 0 or past the end: none
    const bool whole = v >= 0 && v + kVec <= p.vocab;
    float z[kVec];
    if (vec && whole) {
      load_f32<TI, kVec>(in + v, z);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        z[j] = v + j >= 0 && v + j < p.vocab ? to_f32(in[v + j]) : 0.0f;
    }
    if constexpr (TABLE) {
      const uint4 a = *reinterpret_cast<const uint4*>(table + (w - w0));
      const uint4 b = *reinterpret_cast<const uint4*>(table + (w - w0) + 4);
      const uint32_t word[kVec] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (word[j]) z[j] = adjust(z[j], word[j], v + j, r, p);
      }
    }
    if (mask) {
      uint32_t bits = 0;  // bit j: token v + j may follow
      const int32_t last = (p.vocab - 1) >> 5;
      const int32_t lo = v >> 5;  // (floor: -1 when v < 0)
      const uint32_t word0 = lo >= 0 ? __ldg(mask + lo) : 0u;
      const uint32_t word1 = lo < last && (v & 31) > 32 - kVec ? __ldg(mask + lo + 1) : 0u;
      bits = __funnelshift_r(word0, word1, (uint32_t)(v & 31));
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (!((bits >> j) & 1u)) z[j] = __int_as_float(0xff800000);
    }
    if (vec && whole) {
      store_f32<TO, kVec>(out + v, z);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (v + j >= 0 && v + j < p.vocab) out[v + j] = from_f32<TO>(z[j]);
    }
  }
}

template <typename TI, typename TO, bool TABLE>
cudaError_t launch(const LogitsParams& p, cudaStream_t stream) {
  const size_t smem = TABLE ? (size_t)p.slice * sizeof(uint32_t) : 0;
  auto kernel = logits_kernel<TI, TO, TABLE>;
  if (TABLE) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxSlice * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.rows * p.slices), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename TI, typename TO>
cudaError_t by_table(const LogitsParams& p, cudaStream_t stream) {
  return p.tokens || p.bias_tokens ? launch<TI, TO, true>(p, stream) : launch<TI, TO, false>(p, stream);
}

template <typename TI>
cudaError_t by_out(const LogitsParams& p, int elem_out, cudaStream_t stream) {
  switch (elem_out) {
    case kElemF16: return by_table<TI, __half>(p, stream);
    case kElemBF16: return by_table<TI, __nv_bfloat16>(p, stream);
    case kElemF32: return by_table<TI, float>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_logits(LogitsParams p, int elem_in, int elem_out, int sms, cudaStream_t stream) {
  // Slices as long as the table allows, so that few CTAs read the same history; shorter
  // ones where the rows alone do not give every SM two CTAs.
  const int64_t width = (int64_t)p.vocab + kVec - 1;  // with the largest shift
  const int64_t want = std::max<int64_t>(1, ((int64_t)2 * sms + p.rows - 1) / p.rows);
  int64_t slice = (width + want - 1) / want;
  slice = std::min<int64_t>(std::max<int64_t>(slice, kMinSlice), kMaxSlice);
  const int64_t n = (width + slice - 1) / slice;
  slice = ((width + n - 1) / n + 31) / 32 * 32;  // even slices
  p.slice = (int32_t)slice;
  p.slices = (int32_t)((width + slice - 1) / slice);
  switch (elem_in) {
    case kElemF16: return by_out<__half>(p, elem_out, stream);
    case kElemBF16: return by_out<__nv_bfloat16>(p, elem_out, stream);
    case kElemF32: return by_out<float>(p, elem_out, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gb300

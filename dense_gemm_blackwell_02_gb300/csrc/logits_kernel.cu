// Logits before sampling: for every row i and token v
//     z = logits[i][v];  in the history: z = z > 0 ? z / rep : z * rep
//     c times generated: z -= freq * c + (c > 0 ? pres : 0);  z += biases of v
//     masked out: z = -inf
// in binary32, rounded once.
//
// A handful of operations per element: bound by HBM, one read and one write of the logits.
// A CTA owns one slice of one row's vocabulary.  It counts the row's whole history into a
// table in shared memory, 16 bits per token of its slice (the history is short next to the
// vocabulary and comes from L2 after the row's first slice), then streams its logits past
// the table once.  A row that generated more tokens than 14 bits count goes in two halves
// with 32 bits per token.  Integer counts: the result does not depend on the order of the
// atomics.
//
// 256 x 128256 binary32: 43 us without lists (262 MB at 6.1 TB/s), 59 to 60 us with histories of
// up to 8192 tokens, biases and masks: some lane of nearly every warp meets a token of the
// history, and their entries take 10 us, the biases 3, the masks 2.  37 x 50257 fp16 with 4096
// tokens and 200 biases 12 us, 8.7 without the biases, 3.5 without lists.  Other forms measured: eight CTAs per SM of half the
// size, the same; copying first and then rewriting only the logits that the lists name, 70 us
// (each of the row's slices goes through the history twice); the same from a list of the
// distinct tokens, 65; the row's CTAs as a cluster that counts in distributed shared memory,
// 92 (remote atomics); a warp's listed logits gathered in shared memory at every step and
// adjusted side by side, 84 (its registers spill at three CTAs per SM).
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 512;
constexpr int kOcc = 3;            // CTAs per SM
constexpr int kVec = 8;            // logits per thread and step
constexpr int kTokens = 8;         // history tokens per thread in flight
constexpr int kMaxSlice = 24576;   // tokens per CTA: 48 KiB of table
static_assert(kMaxSlice * 2 <= 48 * 1024, "more would have to be asked for at every launch");
constexpr int kMinSlice = 2048;

// A token's entry in the table: how often it was generated, and two flags; 16 bits or 32.
template <bool WIDE>
struct Entry {
  static constexpr uint32_t kInPrompt = WIDE ? 1u << 31 : 1u << 15;
  static constexpr uint32_t kHasBias = WIDE ? 1u << 30 : 1u << 14;
  static constexpr uint32_t kCount = kHasBias - 1u;
  static __device__ __forceinline__ void add(uint32_t* table, int32_t at) {
    if constexpr (WIDE) atomicAdd(table + at, 1u);
    else atomicAdd(table + (at >> 1), 1u << (16 * (at & 1)));
  }
  static __device__ __forceinline__ void flag(uint32_t* table, int32_t at, uint32_t f) {
    if constexpr (WIDE) atomicOr(table + at, f);
    else atomicOr(table + (at >> 1), f << (16 * (at & 1)));
  }
};

struct RowRules {
  float rep, freq, pres;
  int64_t t0, t1, said;  // the row's history, and where its generated part begins
  int64_t bias0, bias1;
  const uint32_t* mask;
};

// A token's logit through the penalties and biases its entry calls for.  ORDERED: the row's
// biases are in the order of their tokens.
template <bool WIDE, bool ORDERED>
__device__ __forceinline__ float adjust(float z, uint32_t entry, int32_t v, const RowRules& r,
                                        const LogitsParams& p) {
  using E = Entry<WIDE>;
  if (entry & ~E::kHasBias) {
    z = z > 0.0f ? __fdiv_rn(z, r.rep) : z * r.rep;
    const uint32_t c = entry & E::kCount;
    if (c) z = z - r.freq * (float)c - r.pres;
  }
  if (entry & E::kHasBias) {
    float w = 0.0f;
    if constexpr (ORDERED) {
      int64_t lo = r.bias0, hi = r.bias1;  // the first of the token's
      while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (p.bias_tokens[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      for (; lo < r.bias1 && p.bias_tokens[lo] == v; ++lo) w += p.bias_values[lo];
    } else {
      for (int64_t i = r.bias0; i < r.bias1; ++i)
        if (p.bias_tokens[i] == v) w += p.bias_values[i];
    }
    z += w;
  }
  return z;
}

// The logits of positions w0..w1-1 of a row (see do_slice) past the table; `next` holds the
// thread's first whole vector.
template <typename TI, typename TO, bool TABLE, bool WIDE, bool ORDERED>
__device__ __forceinline__ void stream(const LogitsParams& p, const RowRules& r, const TI* in, TO* out,
                                       int32_t shift, bool vec, int32_t w0, int32_t w1,
                                       const uint32_t* table, Pack<TI, kVec> next) {
  auto whole = [&](int32_t w) { return w >= shift && w - shift + kVec <= p.vocab; };
  for (int32_t w = w0 + (int32_t)threadIdx.x * kVec; w < w1; w += kThreads * kVec) {
    const int32_t v = w - shift;  // the first of kVec tokens; below 0 or past the end: none
    float z[kVec];
    if (vec && whole(w)) {
      unpack(next, z);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        z[j] = v + j >= 0 && v + j < p.vocab ? to_f32(in[v + j]) : 0.0f;
    }
    const int32_t ahead = w + kThreads * kVec;
    if (vec && ahead < w1 && whole(ahead))
      next = *reinterpret_cast<const Pack<TI, kVec>*>(in + ahead - shift);
    if constexpr (TABLE) {
      if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const uint32_t entry = table[w - w0 + j];
          if (entry) z[j] = adjust<WIDE, ORDERED>(z[j], entry, v + j, r, p);
        }
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(table + (w - w0) / 2);
        if (a.x | a.y | a.z | a.w) {
          const uint32_t two[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            const uint32_t entry = (two[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
            if (entry) z[j] = adjust<WIDE, ORDERED>(z[j], entry, v + j, r, p);
          }
        }
      }
    }
    if (r.mask) {
      // bit j: token v + j may follow
      const int32_t last = (p.vocab - 1) >> 5;
      const int32_t lo = v >> 5;  // (floor: -1 when v < 0)
      const uint32_t word0 = lo >= 0 ? __ldg(r.mask + lo) : 0u;
      const uint32_t word1 = lo < last && (v & 31) > 32 - kVec ? __ldg(r.mask + lo + 1) : 0u;
      const uint32_t bits = __funnelshift_r(word0, word1, (uint32_t)(v & 31));
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (!((bits >> j) & 1u)) z[j] = __int_as_float(0xff800000);
    }
    if (vec && whole(w)) {
      store_f32<TO, kVec>(out + v, z);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (v + j >= 0 && v + j < p.vocab && w + j < w1) out[v + j] = from_f32<TO>(z[j]);
    }
  }
}

// The same for biases in any order: searched through from end to end.  Not inlined, so that it
// takes nothing from the usual case (a flag that chose between the searches spilled there, and
// a search behind a call took 97 us where 59 stayed).
template <typename TI, typename TO, bool WIDE>
__device__ __noinline__ void stream_unordered(const LogitsParams& p, RowRules r, const TI* in, TO* out,
                                              int32_t shift, bool vec, int32_t w0, int32_t w1,
                                              const uint32_t* table) {
  Pack<TI, kVec> next;
  const int32_t first = w0 + (int32_t)threadIdx.x * kVec;
  if (vec && first < w1 && first >= shift && first - shift + kVec <= p.vocab)
    next = *reinterpret_cast<const Pack<TI, kVec>*>(in + first - shift);
  stream<TI, TO, true, WIDE, false>(p, r, in, out, shift, vec, w0, w1, table, next);
}

// Positions w0..w1-1 of a row (w0 a multiple of kVec; position w is token w - shift): the
// table, then the logits.
template <typename TI, typename TO, bool TABLE, bool WIDE>
__device__ __forceinline__ void do_slice(const LogitsParams& p, const RowRules& r, const TI* in,
                                         TO* out, int32_t shift, bool vec, int32_t w0, int32_t w1,
                                         uint32_t* table) {
  // The first logits are on their way while the table is built, and every step's while the
  // one before is worked on; kept as loaded.
  auto whole = [&](int32_t w) { return w >= shift && w - shift + kVec <= p.vocab; };
  Pack<TI, kVec> next;
  const int32_t first = w0 + (int32_t)threadIdx.x * kVec;
  if (vec && first < w1 && whole(first)) next = *reinterpret_cast<const Pack<TI, kVec>*>(in + first - shift);

  if constexpr (TABLE) {
    uint4* t4 = reinterpret_cast<uint4*>(table);
    const int32_t quads = (w1 - w0 + (WIDE ? 3 : 7)) / (WIDE ? 4 : 8);
    for (int32_t i = (int32_t)threadIdx.x; i < quads; i += kThreads) t4[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const uint32_t lo = (uint32_t)max(w0 - shift, 0), hi = (uint32_t)(w1 - shift);  // its tokens
    for (int64_t i0 = r.t0 + threadIdx.x; i0 < r.t1; i0 += kThreads * kTokens) {
      uint32_t v[kTokens];
#pragma unroll
      for (int j = 0; j < kTokens; ++j)
        v[j] = i0 + j * kThreads < r.t1 ? (uint32_t)__ldg(p.tokens + i0 + j * kThreads) : 0xFFFFFFFFu;
#pragma unroll
      for (int j = 0; j < kTokens; ++j) {
        if (v[j] < lo || v[j] >= hi) continue;  // padding, or another slice's
        const int32_t at = (int32_t)v[j] + shift - w0;
        if (i0 + j * kThreads >= r.said) Entry<WIDE>::add(table, at);
        else Entry<WIDE>::flag(table, at, Entry<WIDE>::kInPrompt);
      }
    }
    int falls = 0;
    for (int64_t i = r.bias0 + threadIdx.x; i < r.bias1; i += kThreads) {
      const int32_t token = __ldg(p.bias_tokens + i);
      const uint32_t v = (uint32_t)token;
      if (v >= lo && v < hi) Entry<WIDE>::flag(table, (int32_t)v + shift - w0, Entry<WIDE>::kHasBias);
      if (i > r.bias0 && __ldg(p.bias_tokens + i - 1) > token) falls = 1;
    }
    if (__syncthreads_or(falls)) {
      stream_unordered<TI, TO, WIDE>(p, r, in, out, shift, vec, w0, w1, table);
      return;
    }
  }
  stream<TI, TO, TABLE, WIDE, true>(p, r, in, out, shift, vec, w0, w1, table, next);
}

// TABLE: there are histories or biases to look up.
template <typename TI, typename TO, bool TABLE>
__global__ void __launch_bounds__(kThreads, kOcc) logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ __align__(16) uint32_t table[];
  grid_dependency_wait();
  grid_launch_dependents();

  const int32_t row = (int32_t)(blockIdx.x / (uint32_t)p.slices);
  const int32_t part = (int32_t)(blockIdx.x - (uint32_t)row * (uint32_t)p.slices);
  const TI* in = static_cast<const TI*>(p.in) + (int64_t)row * p.in_stride;
  TO* out = static_cast<TO*>(p.out) + (int64_t)row * p.out_stride;
  // Rows of any alignment: positions are counted from the boundary of kVec elements below
  // the row's start, w = v + shift, so that vectors of positions are aligned (in input and
  // output alike, else single elements are moved).
  const int32_t shift = (int32_t)((reinterpret_cast<uintptr_t>(in) / sizeof(TI)) % kVec);
  const bool vec = (int32_t)((reinterpret_cast<uintptr_t>(out) / sizeof(TO)) % kVec) == shift;
  const int32_t w0 = part * p.slice, w1 = min(w0 + p.slice, p.vocab + shift);
  if (w0 >= w1) return;  // (the last slice of a row with a small shift)

  RowRules r{1.0f, 0.0f, 0.0f, 0, 0, 0, 0, 0, nullptr};
  if (p.tokens) {
    r.t0 = p.token_start[row];
    r.t1 = p.token_start[row + 1];
    r.said = r.t0 + (p.prompt_len ? p.prompt_len[row] : 0);
    if (p.repetition) r.rep = p.repetition[row];
    if (p.frequency) r.freq = p.frequency[row];
    if (p.presence) r.pres = p.presence[row];
  }
  if (p.bias_tokens) {
    r.bias0 = p.bias_start[row];
    r.bias1 = p.bias_start[row + 1];
  }
  if (p.mask) {
    const int64_t m = p.mask_row ? p.mask_row[row] : row;
    if (m >= p.mask_count) {
      if (threadIdx.x == 0) record_bad_index(p.status, kSiteMaskRow);
    } else if (m >= 0) {
      r.mask = p.mask + m * p.mask_stride;
    }
  }
  if (!TABLE || r.t1 - r.said <= (int64_t)Entry<false>::kCount) {
    do_slice<TI, TO, TABLE, false>(p, r, in, out, shift, vec, w0, w1, table);
  } else {
    const int32_t mid = min(w0 + p.slice / 2, w1);
    do_slice<TI, TO, TABLE, true>(p, r, in, out, shift, vec, w0, mid, table);
    __syncthreads();
    if (mid < w1) do_slice<TI, TO, TABLE, true>(p, r, in, out, shift, vec, mid, w1, table);
  }
}

template <typename TI, typename TO, bool TABLE>
cudaError_t launch(const LogitsParams& p, cudaStream_t stream) {
  const size_t smem = TABLE ? (size_t)p.slice * 2 : 0;
  auto kernel = logits_kernel<TI, TO, TABLE>;
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
  // Slices as long as the table allows; shorter ones where the rows alone do not give every
  // SM two CTAs.
  const int64_t width = (int64_t)p.vocab + kVec - 1;  // with the largest shift
  const int64_t want = std::max<int64_t>(1, ((int64_t)2 * sms + p.rows - 1) / p.rows);
  int64_t slice = (width + want - 1) / want;
  slice = std::min<int64_t>(std::max<int64_t>(slice, kMinSlice), kMaxSlice);
  int64_t n = (width + slice - 1) / slice;
  p.slice = (int32_t)(((width + n - 1) / n + 63) / 64 * 64);  // even slices, of even halves
  p.slices = (int32_t)((width + p.slice - 1) / p.slice);
  switch (elem_in) {
    case kElemF16: return by_out<__half>(p, elem_out, stream);
    case kElemBF16: return by_out<__nv_bfloat16>(p, elem_out, stream);
    case kElemF32: return by_out<float>(p, elem_out, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gb300

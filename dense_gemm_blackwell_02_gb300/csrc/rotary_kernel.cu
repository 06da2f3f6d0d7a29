// Rotary positions with several axes: pair i of every head of token t turns by the angle
// theta = theta_i(positions[axis(i)][t]), whose cosine and sine come from tables:
//     a' = a cos - b sin,  b' = b cos + a sin          (the inverse negates sin)
// in binary32, rounded once to the element type.
//
// Six operations per pair against 4 elements moved: bound by HBM, so the kernel is one
// pass of 16-byte accesses.  A CTA takes the heads of a few tokens.  It first gathers the
// tokens' cosines and sines, pair by pair from the rows that the pairs' axes ask for, into
// shared memory, while the first elements are already on their way; then every thread owns
// one vector of pairs of a head (two vectors of the head when a pair's halves lie apart, one
// when they are neighbours) and walks the heads, several loads in flight.
//
// Measured over cold operands: 8192 tokens x 72 heads x 128, bf16, 52 to 53 us (302 MB at 5.8
// TB/s, 0.86 of a copy's rate); 4099 x 16 x 80 binary32, neighbours, 11.5 us (43 MB at 3.7 TB/s:
// a second round of CTAs would be short, so the tokens per CTA are chosen for one); 256 x 72 x
// 128 bf16 4.7 us and one token 2.3, both a launch and one trip to memory.  With the tables
// read from L2 for every head and one head's loads in flight the first took 80 us.  Halves that
// are no whole vectors move single elements: 8192 x 16 x 72 bf16 26.8 us, of 80 with 40 turned 43.
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 256;
constexpr int kRun = 3;         // heads whose loads are in flight together, per thread
constexpr int kMaxTokens = 8;   // tokens per CTA at most

// N neighbouring values of the table (16-byte aligned for N >= 4, 8-byte for 2).
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&f)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + j);
      f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x, f[1] = v.y;
  } else {
    f[0] = *p;
  }
}

// A CTA's tokens and heads.
struct Share {
  int32_t t0, nt, h0, nh;
  __device__ __forceinline__ explicit Share(const RotaryParams& p) {
    const int32_t tile = (int32_t)(blockIdx.x / (uint32_t)p.shares);
    const int32_t share = (int32_t)(blockIdx.x - (uint32_t)tile * (uint32_t)p.shares);
    t0 = tile * p.tile_tokens, nt = min(p.tile_tokens, p.tokens - t0);
    h0 = share * p.share_heads, nh = min(p.share_heads, p.heads - h0);
  }
};

// The CTA's heads, pair by pair, for tokens with a position outside the tables: those pairs
// stay as they are, infinities and NaN included, which a turn by no angle would not leave.
template <typename T, bool NEIGH>
__device__ __noinline__ void one_by_one(const RotaryParams& p, const float* table) {
  const Share at(p);
  const int t0 = at.t0, nt = at.nt, nh = at.nh;
  const T* x = static_cast<const T*>(p.x) + (int64_t)t0 * p.x_token + (int64_t)at.h0 * p.x_head;
  T* y = static_cast<T*>(p.y) + (int64_t)t0 * p.y_token + (int64_t)at.h0 * p.y_head;
  const int per_head = p.half + (static_cast<const void*>(p.x) == p.y ? 0 : p.dim - 2 * p.half);
  const int64_t all = (int64_t)nt * nh * per_head;
  for (int64_t i = threadIdx.x; i < all; i += kThreads) {
    const int64_t r = i / per_head;
    const int e = (int)(i - r * per_head), t = (int)(r / nh), h = (int)(r - (int64_t)t * nh);
    const T* from = x + t * p.x_token + h * p.x_head;
    T* to = y + t * p.y_token + h * p.y_head;
    if (e >= p.half) {  // past the pairs
      to[e + p.half] = from[e + p.half];
      continue;
    }
    const int ia = NEIGH ? 2 * e : e, ib = NEIGH ? 2 * e + 1 : e + p.half;
    const T a = from[ia], b = from[ib];
    const int64_t pos = p.positions[(int64_t)p.pair_axis[e] * p.tokens + t0 + t];
    if (pos < 0 || pos >= p.num_positions) {
      to[ia] = a;
      to[ib] = b;
      continue;
    }
    const float u = to_f32(a), v = to_f32(b);
    const float c = table[t * 2 * p.half + e], s = table[t * 2 * p.half + p.half + e];
    to[ia] = from_f32<T>(u * c - v * s);
    to[ib] = from_f32<T>(v * c + u * s);
  }
}

// NEIGH: neighbouring pairs.  V: elements per vector (1: no alignment is assumed).
template <typename T, bool NEIGH, int V>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryParams p) {
  // pairs per item: V with the halves apart (two vectors), V / 2 as neighbours (one; with
  // V = 1 two single elements)
  constexpr int kPairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  constexpr int kSpan = NEIGH ? 2 * kPairs : V;  // elements of one access
  extern __shared__ __align__(16) float table[];  // per token: half cosines, half sines
  grid_dependency_wait();
  grid_launch_dependents();

  const Share at_share(p);
  const int32_t t0 = at_share.t0, nt = at_share.nt, h0 = at_share.h0, nh = at_share.nh;
  const int lanes = min(p.items, kThreads);   // threads per head
  const int groups = kThreads / lanes;        // heads at a time
  const int g = (int)threadIdx.x / lanes;
  const int pair_items = p.half / kPairs;
  const T* x = static_cast<const T*>(p.x) + (int64_t)t0 * p.x_token + (int64_t)h0 * p.x_head;
  T* y = static_cast<T*>(p.y) + (int64_t)t0 * p.y_token + (int64_t)h0 * p.y_head;
  const int rows = nt * nh;                   // heads of all tokens
  // A thread's heads are `groups` apart: tokens and heads onward, and back at a token's end.
  const int step_t = groups / nh, step_h = groups - step_t * nh;
  struct Cursor {
    const T* x;
    T* y;
    int t, h, r;
  };
  auto advance = [&](Cursor& c) {
    c.r += groups;
    c.t += step_t;
    c.h += step_h;
    c.x += step_t * p.x_token + step_h * p.x_head;
    c.y += step_t * p.y_token + step_h * p.y_head;
    if (c.h >= nh) {
      c.h -= nh;
      ++c.t;
      c.x += p.x_token - nh * p.x_head;
      c.y += p.y_token - nh * p.y_head;
    }
  };
  Pack<T, kSpan> a[kRun], b[kRun];

  // The next kRun heads of an item, as loaded ...
  auto load = [&](int item, Cursor c) {
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (c.r >= rows) break;
      if (item >= pair_items) {  // past the pairs: copied
        *reinterpret_cast<Pack<T, V>*>(&a[k]) =
            *reinterpret_cast<const Pack<T, V>*>(c.x + 2 * p.half + (item - pair_items) * V);
      } else if constexpr (NEIGH && V == 1) {
        a[k].v[0] = c.x[2 * item];
        a[k].v[1] = c.x[2 * item + 1];
      } else {
        a[k] = *reinterpret_cast<const Pack<T, kSpan>*>(c.x + item * kSpan);
        if constexpr (!NEIGH) b[k] = *reinterpret_cast<const Pack<T, kSpan>*>(c.x + item * kSpan + p.half);
      }
      advance(c);
    }
  };
  // ... and turned; the cursor moves on.
  auto finish = [&](int item, Cursor& c) {
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (c.r >= rows) break;
      if (item >= pair_items) {
        *reinterpret_cast<Pack<T, V>*>(c.y + 2 * p.half + (item - pair_items) * V) =
            *reinterpret_cast<const Pack<T, V>*>(&a[k]);
        advance(c);
        continue;
      }
      const float* row = table + c.t * 2 * p.half + item * kPairs;
      float cs[kPairs], sn[kPairs];
      load_row<kPairs>(row, cs);
      load_row<kPairs>(row + p.half, sn);
      T* at = c.y + item * kSpan;
      if constexpr (NEIGH) {
        float in[kSpan], o[kSpan];
        if constexpr (V == 1) in[0] = to_f32(a[k].v[0]), in[1] = to_f32(a[k].v[1]);
        else unpack(a[k], in);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float u = in[2 * j], v = in[2 * j + 1];
          o[2 * j] = u * cs[j] - v * sn[j];
          o[2 * j + 1] = v * cs[j] + u * sn[j];
        }
        if constexpr (V == 1) {
          at[0] = from_f32<T>(o[0]);
          at[1] = from_f32<T>(o[1]);
        } else {
          store_f32<T, kSpan>(at, o);
        }
      } else {
        float u[kSpan], v[kSpan], oa[kSpan], ob[kSpan];
        unpack(a[k], u);
        unpack(b[k], v);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          oa[j] = u[j] * cs[j] - v[j] * sn[j];
          ob[j] = v[j] * cs[j] + u[j] * sn[j];
        }
        store_f32<T, kSpan>(at, oa);
        store_f32<T, kSpan>(at + p.half, ob);
      }
      advance(c);
    }
  };
  Cursor start;
  start.r = g;
  start.t = g / nh;
  start.h = g - start.t * nh;
  start.x = x + start.t * p.x_token + start.h * p.x_head;
  start.y = y + start.t * p.y_token + start.h * p.y_head;

  const bool works = g < groups;
  int item = (int)threadIdx.x - g * lanes;
  // (in place there is nothing to do past the pairs)
  const int items = static_cast<const void*>(p.x) == p.y ? pair_items : p.items;
  if (works && item < items) load(item, start);
  int outside = 0;
  for (int i = (int)threadIdx.x; i < nt * p.half; i += kThreads) {
    const int t = i / p.half, pair = i - t * p.half;
    const int64_t pos = p.positions[(int64_t)p.pair_axis[pair] * p.tokens + t0 + t];
    float c = 1.0f, s = 0.0f;
    if (pos >= 0 && pos < p.num_positions) {
      c = __ldg(p.cos + pos * p.half + pair);
      s = __ldg(p.sin + pos * p.half + pair);
    } else {
      record_bad_index(p.status, kSitePosition);
      outside = 1;
    }
    table[t * 2 * p.half + pair] = c;
    table[t * 2 * p.half + p.half + pair] = p.inverse ? -s : s;
  }
  if (__syncthreads_or(outside)) {
    one_by_one<T, NEIGH>(p, table);
    return;
  }
  if (!works) return;
  for (; item < items; item += lanes) {
    Cursor c = start;
    while (c.r < rows) {
      if (c.r != g || item >= lanes) load(item, c);
      finish(item, c);
    }
  }
}

template <typename T, bool NEIGH, int V>
cudaError_t launch(RotaryParams& p, int sms, cudaStream_t stream) {
  const int pairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  p.items = p.half / pairs + (p.dim - 2 * p.half) / V;
  const int groups = kThreads / std::min(p.items, kThreads);
  // A CTA takes as many tokens as give every thread three runs of heads, as long as every
  // SM has two CTAs; with fewer tokens than that, shares of one token's heads.  (8192 x 72 x
  // 128 bf16: one run 70 us, two 55.6, three 53.1, six 58.9.  256 x 72 x 128: 4.6 us, with
  // smaller CTAs, eight to an SM, 6.3.)
  const int64_t want = (int64_t)3 * kRun * groups;  // heads per CTA
  const int64_t spread = ((int64_t)p.tokens * p.heads + 2 * sms - 1) / (2 * sms);
  const int64_t per_cta = std::max<int64_t>(groups, std::min(want, spread));
  p.tile_tokens = (int32_t)std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, per_cta / p.heads));
  // (four CTAs per SM are resident: not a second round of a few CTAs after a full first one;
  // 4099 x 16 x 80 binary32 in 684 CTAs 14.2 us, in 586 11.9)
  const int64_t resident = (int64_t)4 * sms;
  if ((p.tokens + p.tile_tokens - 1) / p.tile_tokens <= resident * 3 / 2)
    p.tile_tokens = (int32_t)std::min<int64_t>(
        kMaxTokens, std::max<int64_t>(p.tile_tokens, (p.tokens + resident - 1) / resident));
  p.shares = (int32_t)((p.heads + per_cta - 1) / per_cta);
  p.share_heads = (p.heads + p.shares - 1) / p.shares;
  p.shares = (p.heads + p.share_heads - 1) / p.share_heads;
  const int64_t tiles = ((int64_t)p.tokens + p.tile_tokens - 1) / p.tile_tokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * p.shares), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)p.tile_tokens * 2 * p.half * sizeof(float);
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

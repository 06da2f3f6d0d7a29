// Normed query and key heads with their rotary positions, in one pass, and the gradients.  For
// every head x of `dim` values with weights w (the query heads' or the key heads'):
//     r = 1 / sqrt(sum x^2 / dim + eps),   n = x r w,   y = R n
// R turns pair i by the angle of its token's position (as in rotary_kernel.cu).  Backwards, with
// dn = R^T dy (the inverse turn) and g = dn w:
//     dx = r g - x (r^3 / dim) sum g x,     dw = sum over tokens and heads of dn x r
// in binary32, rounded once to the element type; dw stays binary32.
//
// One read and one write per element (backwards two reads), a dozen operations: bound by HBM.  A
// head lies in the registers of a few neighbouring lanes, the two halves of its pairs in the same
// lane, so that its sum takes one reduction over those lanes and nothing is read twice.  What the
// heads of a token share waits in shared memory, in an order that neighbouring lanes read without
// bank conflicts (Chunks): forwards the products of weights, cosines and sines (so that a pair
// takes four multiplications and two by r), backwards both apart.  Two instructions' worth of
// binary32 are issued as one (f32x2), and the next heads are on their way while one is worked on.
// Backwards, a CTA walks its share of the tokens with the query heads or with
// the key heads and keeps its sums for dw in registers; a second kernel adds the CTAs' sums in
// their order, so that the result is the same from run to run.
//
// Measured: forwards 8192 x 72 x 128 bf16 56 us (5.4 TB/s, a copy's 6.8), backwards 102 (4.4 TB/s;
// 16 warps per SM, which this layout's registers allow, fill neither memory nor issue); 4099 x 16 x
// 80 fp32 21, of which the second kernel takes 3; one token 2.9, a launch and two trips to memory.
#pragma once
#include <algorithm>
#include <cstring>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs per SM, for lanes that hold so many accesses of a head
constexpr int heads_per_sm(int per_lane, bool back) { return !back ? (per_lane == 1 ? 3 : 2) : per_lane <= 2 ? 2 : 1; }

// Two operations in one instruction, each rounded as the single one.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a_, b_, d_;\n\tmov.b64 a_, {%2, %3};\n\tmov.b64 b_, {%4, %5};\n\t"
      "mul.rn.f32x2 d_, a_, b_;\n\tmov.b64 {%0, %1}, d_;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a_, b_, c_, d_;\n\tmov.b64 a_, {%2, %3};\n\tmov.b64 b_, {%4, %5};\n\t"
      "mov.b64 c_, {%6, %7};\n\tfma.rn.f32x2 d_, a_, b_, c_;\n\tmov.b64 {%0, %1}, d_;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
// Of N values each: d = a b, d = a b + c.
template <int N>
__device__ __forceinline__ void mul_each(float* d, const float* a, const float* b) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int j = 0; j < N; j += 2) mul2(d[j], d[j + 1], a[j], a[j + 1], b[j], b[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) d[j] = a[j] * b[j];
  }
}
template <int N>
__device__ __forceinline__ void mul_all(float* d, const float* a, float b) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int j = 0; j < N; j += 2) mul2(d[j], d[j + 1], a[j], a[j + 1], b, b);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) d[j] = a[j] * b;
  }
}
template <int N>
__device__ __forceinline__ void fma_each(float* d, const float* a, const float* b, const float* c) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int j = 0; j < N; j += 2) fma2(d[j], d[j + 1], a[j], a[j + 1], b[j], b[j + 1], c[j], c[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) d[j] = fmaf(a[j], b[j], c[j]);
  }
}
template <int N>
__device__ __forceinline__ void fma_all(float* d, const float* a, float b, const float* c) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int j = 0; j < N; j += 2) fma2(d[j], d[j + 1], a[j], a[j + 1], b, b, c[j], c[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) d[j] = fmaf(a[j], b, c[j]);
  }
}

// N values for each of `items` items in shared memory, as chunks of 16 (or 8, or 4) bytes, all
// items' first chunks before their second ones: lanes with neighbouring items read neighbouring
// chunks.
template <int N>
struct Chunks {
  static constexpr int kWide = N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
  static __device__ __forceinline__ int at(int e, int item, int items) {
    return (e / kWide * items + item) * kWide + e % kWide;
  }
  static __device__ __forceinline__ void load(const float* base, int item, int items, float (&f)[N]) {
#pragma unroll
    for (int c = 0; c < N / kWide; ++c) {
      const float* p = base + (c * items + item) * kWide;
      if constexpr (kWide == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[4 * c] = v.x, f[4 * c + 1] = v.y, f[4 * c + 2] = v.z, f[4 * c + 3] = v.w;
      } else if constexpr (kWide == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[2 * c] = v.x, f[2 * c + 1] = v.y;
      } else {
        f[c] = *p;
      }
    }
  }
};

__device__ __forceinline__ float weight_at(const void* w, int elem, int i) {
  if (!w) return 1.0f;
  if (elem == kElemF32) return static_cast<const float*>(w)[i];
  if (elem == kElemF16) return __half2float(static_cast<const __half*>(w)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// How a lane holds its part of a head.  V: elements per access (1: no alignment is assumed); a
// pair item is V pairs in two vectors half the turned values apart or, NEIGH, V / 2 pairs in one
// (V = 1: one pair, two accesses); the items behind the pairs are V values each.
template <typename T, bool NEIGH, int V>
struct Item {
  static constexpr int kPairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  static constexpr int kSpan = NEIGH ? 2 * kPairs : V;
  Pack<T, kSpan> a, b;  // (b: the second halves, unless NEIGH)

  __device__ __forceinline__ void load(const T* row, int item, int pair_items, int half) {
    if (item >= pair_items) {
      *reinterpret_cast<Pack<T, V>*>(&a) =
          *reinterpret_cast<const Pack<T, V>*>(row + 2 * half + (item - pair_items) * V);
    } else if constexpr (NEIGH && V == 1) {
      a.v[0] = row[2 * item];
      a.v[1] = row[2 * item + 1];
    } else {
      a = *reinterpret_cast<const Pack<T, kSpan>*>(row + item * kSpan);
      if constexpr (!NEIGH) b = *reinterpret_cast<const Pack<T, kSpan>*>(row + item * kSpan + half);
    }
  }
  // The same by way of shared memory (16-byte accesses): asked for there ...
  static constexpr int kVectors = NEIGH ? 1 : 2;
  static __device__ __forceinline__ void ask(uint32_t to, uint32_t step, const T* row, int item, int pair_items,
                                             int half) {
    if (item >= pair_items) {
      cp_async_cg_16(to, row + 2 * half + (item - pair_items) * V);
    } else {
      cp_async_cg_16(to, row + item * kSpan);
      if constexpr (!NEIGH) cp_async_cg_16(to + step, row + item * kSpan + half);
    }
  }
  // ... and taken.
  __device__ __forceinline__ void take(uint32_t from, uint32_t step) {
    const uint4 v = ld_shared_v4(from);
    memcpy(&a, &v, 16);
    if constexpr (!NEIGH) {
      const uint4 w = ld_shared_v4(from + step);
      memcpy(&b, &w, 16);
    }
  }
  // As binary32: 2 kPairs values, the first of the pairs and the second ones, or V values and
  // zeros.
  __device__ __forceinline__ void values(bool pairs, float (&f)[2 * kPairs]) const {
    if (!pairs) {
      float x[V];
      unpack(*reinterpret_cast<const Pack<T, V>*>(&a), x);
#pragma unroll
      for (int j = 0; j < 2 * kPairs; ++j) f[j] = j < V ? x[j] : 0.0f;
    } else if constexpr (NEIGH) {
      float x[kSpan];
      unpack(a, x);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) f[j] = x[2 * j], f[kPairs + j] = x[2 * j + 1];
    } else {
      float x[kSpan], z[kSpan];
      unpack(a, x);
      unpack(b, z);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) f[j] = x[j], f[kPairs + j] = z[j];
    }
  }
  static __device__ __forceinline__ void store(T* row, int item, int pair_items, int half,
                                               const float (&f)[2 * kPairs]) {
    if (item >= pair_items) {
      float x[V];
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = f[j];
      store_f32<T, V>(row + 2 * half + (item - pair_items) * V, x);
    } else if constexpr (NEIGH) {
      float x[kSpan];
#pragma unroll
      for (int j = 0; j < kPairs; ++j) x[2 * j] = f[j], x[2 * j + 1] = f[kPairs + j];
      if constexpr (V == 1) {
        row[2 * item] = from_f32<T>(x[0]);
        row[2 * item + 1] = from_f32<T>(x[1]);
      } else {
        store_f32<T, kSpan>(row + item * kSpan, x);
      }
    } else {
      float x[kSpan], z[kSpan];
#pragma unroll
      for (int j = 0; j < kPairs; ++j) x[j] = f[j], z[j] = f[kPairs + j];
      store_f32<T, kSpan>(row + item * kSpan, x);
      store_f32<T, kSpan>(row + item * kSpan + half, z);
    }
  }
};

// Where value j of an item (Item::values) is in the head, -1: nowhere.
template <bool NEIGH, int V>
__device__ __forceinline__ int place_of(int item, int j, int pair_items, int half, int dim) {
  constexpr int kPairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  if (item >= pair_items) {
    const int e = 2 * half + (item - pair_items) * V + j;
    return j < V && e < dim ? e : -1;
  }
  const int pair = item * kPairs + (j < kPairs ? j : j - kPairs);
  if constexpr (NEIGH) return 2 * pair + (j < kPairs ? 0 : 1);
  else return j < kPairs ? pair : pair + half;
}

// The sum over the `lanes` neighbouring lanes of a head, of which this one is number `at` (the
// first at lane `lead`).  Every lane of the warp takes part.
__device__ __forceinline__ float head_sum(float v, int lanes, int at, int lead) {
  if ((lanes & (lanes - 1)) == 0) {
    for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
  }
  for (int off = 16; off > 0; off >>= 1) {
    if (off >= lanes) continue;
    const float o = __shfl_down_sync(0xFFFFFFFFu, v, off);
    if (at + off < lanes) v += o;
  }
  return __shfl_sync(0xFFFFFFFFu, v, lead);
}

// A lane's walk over rows (heads of tokens) `groups` apart.
template <typename T>
struct Cursor {
  const T* x;
  const T* dy;
  T* y;
  int t, h, r;
};

// Shared memory of a CTA, in values: backwards the weights of both kinds of heads for every item,
// forwards of the items behind the pairs only; per token what its pairs are multiplied by,
// forwards for both kinds of heads (weight times cosine and sine, of either value), backwards
// cosines and sines; and whether a pair's position is missing.
template <bool NEIGH, int V, bool BACK>
struct HeadsLayout {
  static constexpr int kPairs = NEIGH ? (V > 1 ? V / 2 : 1) : V;
  static constexpr int kVals = 2 * kPairs;
  static constexpr int kTurn = BACK ? 2 * kPairs : 4 * kPairs;  // per pair item, token (and kind)
  static __host__ __device__ __forceinline__ int weights(int items, int pair_items) {
    return BACK ? items * kVals : (items - pair_items) * V;     // of one kind of heads
  }
  static __host__ __device__ __forceinline__ int turns(int pair_items) { return (BACK ? 1 : 2) * pair_items * kTurn; }
};

// Rows of a lane that wait in shared memory or are on their way there, where they come in 16-byte
// accesses: the one worked on, and as many more as keep about 100 KB per SM in flight without
// registers for them (with one row ahead in registers 8192 x 72 x 128 took 84 us).
template <typename T, bool NEIGH, int V, int I, bool BACK>
constexpr int ring_slots() {
  return V * sizeof(T) != 16 ? 0 : I > 1 ? 3 : BACK ? 4 : 5;
}
template <typename T, bool NEIGH, int V, int I, bool BACK>
constexpr int ring_bytes() {  // of a thread
  return ring_slots<T, NEIGH, V, I, BACK>() * I * (NEIGH ? 1 : 2) * (BACK ? 2 : 1) * 16;
}

template <typename T, bool NEIGH, int V, int I, bool BACK>
__global__ void __launch_bounds__(kThreads, heads_per_sm(I, BACK))
    heads_kernel(const __grid_constant__ HeadsParams p) {
  using It = Item<T, NEIGH, V>;
  using L = HeadsLayout<NEIGH, V, BACK>;
  constexpr int kPairs = L::kPairs, kVals = L::kVals, kTurn = L::kTurn;
  constexpr int kSlots = ring_slots<T, NEIGH, V, I, BACK>();
  extern __shared__ __align__(16) float shared[];
  const int pair_items = p.half / kPairs;
  const int turns = L::turns(pair_items), one_weights = L::weights(p.items, pair_items);
  constexpr int kRing = kThreads * ring_bytes<T, NEIGH, V, I, BACK>();
  float* table = shared + kRing / 4;
  float* weights = table + max(p.tile_tokens, p.key_tile_tokens) * turns;
  uint8_t* unturned = reinterpret_cast<uint8_t*>(weights + 2 * one_weights);
  grid_dependency_wait();
  grid_launch_dependents();

  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int in_warp = 32 / p.lanes;                        // heads of a warp at a time
  const int sub = lane / p.lanes, at = lane - sub * p.lanes;
  const bool works = sub < in_warp;
  const int groups = in_warp * kWarps;
  const int g = warp * in_warp + sub;

  // This CTA's heads and tokens: forwards one tile of tokens with a share of the heads,
  // backwards every step-th tile with the query or the key heads.
  const int set = BACK && (int)blockIdx.x >= p.query_ctas ? 1 : 0;
  int h0, nh, tile, step;
  const int tile_tokens = BACK && set ? p.key_tile_tokens : p.tile_tokens;
  if constexpr (BACK) {
    h0 = set ? p.query_heads : 0;
    nh = set ? p.heads - p.query_heads : p.query_heads;
    tile = (int)blockIdx.x - (set ? p.query_ctas : 0);
    step = set ? (int)gridDim.x - p.query_ctas : p.query_ctas;
  } else {
    tile = (int)(blockIdx.x / (unsigned)p.shares);
    h0 = ((int)blockIdx.x - tile * p.shares) * p.share_heads;
    nh = min(p.share_heads, p.heads - h0);
    step = INT32_MAX / 2;
  }
  // A lane's rows are `groups` apart: tokens and heads onward, and back at a token's end.
  const int step_t = groups / nh, step_h = groups - step_t * nh;
  const int64_t x_step = step_t * p.x_token + step_h * p.x_head, x_wrap = p.x_token - nh * p.x_head;
  const int64_t y_step = step_t * p.y_token + step_h * p.y_head, y_wrap = p.y_token - nh * p.y_head;
  const int64_t dy_step = BACK ? step_t * p.dy_token + step_h * p.dy_head : 0;
  const int64_t dy_wrap = BACK ? p.dy_token - nh * p.dy_head : 0;
  auto advance = [&](Cursor<T>& c) {
    c.r += groups;
    c.t += step_t;
    c.h += step_h;
    c.x += x_step;
    c.y += y_step;
    if constexpr (BACK) c.dy += dy_step;
    if (c.h >= nh) {
      c.h -= nh;
      ++c.t;
      c.x += x_wrap;
      c.y += y_wrap;
      if constexpr (BACK) c.dy += dy_wrap;
    }
  };

  [[maybe_unused]] float dw[I][kVals] = {};
  bool first = true;
  for (int64_t t0 = (int64_t)tile * tile_tokens; t0 < p.tokens; t0 += (int64_t)step * tile_tokens) {
    const int nt = (int)min((int64_t)tile_tokens, p.tokens - t0);
    const int rows = nt * nh;
    struct Row {
      It x[I];
      It dy[BACK ? I : 1];
      T* y;
      int t, h;
      bool on;
    };
    [[maybe_unused]] Row next;
    auto load = [&](const Cursor<T>& c, Row& row) {
      row.on = works && c.r < rows;
      row.y = c.y, row.t = c.t, row.h = c.h;
      if (!row.on) return;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int item = at + i * p.lanes;
        if (item >= p.items) break;
        row.x[i].load(c.x, item, pair_items, p.half);
        if constexpr (BACK) row.dy[i].load(c.dy, item, pair_items, p.half);
      }
    };
    // (a thread's own vectors, a thread after the other: no conflicts, no barriers)
    constexpr uint32_t kStep = kThreads * 16u;
    constexpr uint32_t kItem = It::kVectors * kStep, kSlot = I * (BACK ? 2 : 1) * kItem;
    const uint32_t ring = smem_addr(shared) + threadIdx.x * 16u;
    auto ask = [&](const Cursor<T>& c, int slot) {
      if (works && c.r < rows) {
        const uint32_t to = ring + slot * kSlot;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int item = at + i * p.lanes;
          if (item >= p.items) break;
          It::ask(to + i * kItem, kStep, c.x, item, pair_items, p.half);
          if constexpr (BACK) It::ask(to + (I + i) * kItem, kStep, c.dy, item, pair_items, p.half);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](const Cursor<T>& c, int slot, Row& row) {
      row.on = works && c.r < rows;
      row.y = c.y, row.t = c.t, row.h = c.h;
      const uint32_t from = ring + slot * kSlot;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        row.x[i].take(from + i * kItem, kStep);
        if constexpr (BACK) row.dy[i].take(from + (I + i) * kItem, kStep);
      }
    };
    Cursor<T> c;
    c.r = g;
    c.t = g / nh;
    c.h = g - c.t * nh;
    c.x = static_cast<const T*>(p.x) + (t0 + c.t) * p.x_token + (int64_t)(h0 + c.h) * p.x_head;
    c.y = static_cast<T*>(p.y) + (t0 + c.t) * p.y_token + (int64_t)(h0 + c.h) * p.y_head;
    c.dy = nullptr;
    if constexpr (BACK)
      c.dy = static_cast<const T*>(p.dy) + (t0 + c.t) * p.dy_token + (int64_t)(h0 + c.h) * p.dy_head;
    Cursor<T> ahead = c;
    if constexpr (kSlots > 0) {
#pragma unroll
      for (int k = 0; k < kSlots - 1; ++k) {
        ask(ahead, k);
        advance(ahead);
      }
    } else {
      load(ahead, next);
      advance(ahead);
    }

    if (first) {
      for (int i = (int)threadIdx.x; i < 2 * one_weights; i += kThreads) {
        const int kind = i >= one_weights, j = i - kind * one_weights;
        const void* w = kind ? p.key_weight : p.query_weight;
        if constexpr (BACK) {
          const int item = j / kVals, e = j - item * kVals;
          const int place = place_of<NEIGH, V>(item, e, pair_items, p.half, p.dim);
          weights[kind * one_weights + Chunks<kVals>::at(e, item, p.items)] =
              place < 0 ? 0.0f : weight_at(w, p.weight_elem, place);
        } else {
          weights[i] = weight_at(w, p.weight_elem, 2 * p.half + j);
        }
      }
      first = false;
    }
    int outside = 0;
    // (a few pairs of a thread at a time, so that their loads, each after the other's result, wait
    // together: backwards 8192 x 72 x 128 bf16 154 us one by one, 127 so)
    constexpr int kBatch = BACK ? 4 : 2;
    for (int i0 = (int)threadIdx.x; i0 < nt * p.half; i0 += kBatch * kThreads) {
      int t[kBatch], pair[kBatch];
      int64_t pos[kBatch];
      float cs[kBatch], sn[kBatch];
      bool ok[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = min(i0 + k * kThreads, nt * p.half - 1);
        t[k] = i / p.half, pair[k] = i - t[k] * p.half;
        pos[k] = p.positions[(int64_t)p.pair_axis[pair[k]] * p.tokens + t0 + t[k]];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ok[k] = pos[k] >= 0 && pos[k] < p.num_positions;
        cs[k] = 1.0f, sn[k] = 0.0f;
        if (ok[k]) {
          cs[k] = __ldg(p.cos + pos[k] * p.half + pair[k]);
          sn[k] = __ldg(p.sin + pos[k] * p.half + pair[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kThreads;
        if (i >= nt * p.half) break;
        if (!ok[k]) {
          record_bad_index(p.status, kSitePosition);
          outside = 1;
        }
        unturned[i] = !ok[k];
        const int item = pair[k] / kPairs, j = pair[k] - item * kPairs;
        float* to = table + t[k] * turns;
        if constexpr (BACK) {
          to[Chunks<kTurn>::at(j, item, pair_items)] = cs[k];
          to[Chunks<kTurn>::at(kPairs + j, item, pair_items)] = -sn[k];
        } else {
          const int ia = place_of<NEIGH, V>(item, j, pair_items, p.half, p.dim);
          const int ib = place_of<NEIGH, V>(item, kPairs + j, pair_items, p.half, p.dim);
#pragma unroll
          for (int kind = 0; kind < 2; ++kind, to += pair_items * kTurn) {
            const void* w = kind ? p.key_weight : p.query_weight;
            const float wa = weight_at(w, p.weight_elem, ia), wb = weight_at(w, p.weight_elem, ib);
            to[Chunks<kTurn>::at(j, item, pair_items)] = wa * cs[k];
            to[Chunks<kTurn>::at(kPairs + j, item, pair_items)] = -(wb * sn[k]);
            to[Chunks<kTurn>::at(2 * kPairs + j, item, pair_items)] = wb * cs[k];
            to[Chunks<kTurn>::at(3 * kPairs + j, item, pair_items)] = wa * sn[k];
          }
        }
      }
    }
    const bool any_outside = __syncthreads_or(outside) != 0;

    // (whole warps go through the loop together: the sums are over lanes)
    auto work = [&](const Row& row) {
      const bool on = row.on;
      float f[I][kVals], s = 0.0f;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int item = at + i * p.lanes;
        if (on && item < p.items) {
          row.x[i].values(item < pair_items, f[i]);
        } else {
#pragma unroll
          for (int j = 0; j < kVals; ++j) f[i][j] = 0.0f;
        }
        float sq[kPairs];
        mul_each<kPairs>(sq, f[i], f[i]);
        fma_each<kPairs>(sq, f[i] + kPairs, f[i] + kPairs, sq);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) s += sq[j];
      }
      s = head_sum(s, p.lanes, at, lane - at);
      const float root = __frsqrt_rn(fmaf(s, p.inv_dim, p.eps));
      // (a pair without a position is left as it is, infinities and NaN included)
      auto alone = [&](int item, int j) { return any_outside && unturned[row.t * p.half + item * kPairs + j]; };
      if constexpr (!BACK) {
        const int kind = h0 + row.h < p.query_heads ? 0 : 1;
        const float* turn = table + row.t * turns + kind * pair_items * kTurn;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int item = at + i * p.lanes;
          if (!on || item >= p.items) break;
          mul_all<kVals>(f[i], f[i], root);
          float o[kVals];
          if (item < pair_items) {
            float m[kTurn];
            Chunks<kTurn>::load(turn, item, pair_items, m);
            const float *a = f[i], *b = f[i] + kPairs;
            mul_each<kPairs>(o, a, m);
            mul_each<kPairs>(o + kPairs, b, m + 2 * kPairs);
            if (!any_outside) {
              fma_each<kPairs>(o, b, m + kPairs, o);
              fma_each<kPairs>(o + kPairs, a, m + 3 * kPairs, o + kPairs);
            } else {
#pragma unroll
              for (int j = 0; j < kPairs; ++j)
                if (!alone(item, j)) {
                  o[j] = fmaf(b[j], m[kPairs + j], o[j]);
                  o[kPairs + j] = fmaf(a[j], m[3 * kPairs + j], o[kPairs + j]);
                }
            }
          } else {
            const float* w = weights + kind * one_weights + (item - pair_items) * V;
#pragma unroll
            for (int j = 0; j < kVals; ++j) o[j] = j < V ? f[i][j] * w[j] : 0.0f;
          }
          It::store(row.y, item, pair_items, p.half, o);
        }
      } else {
        const float* w = weights + set * one_weights;
        float gr[I][kVals], along = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int item = at + i * p.lanes;
          if (!on || item >= p.items) break;
          row.dy[i].values(item < pair_items, gr[i]);
          mul_all<kVals>(f[i], f[i], root);  // n
          if (item < pair_items) {
            float m[kTurn], o[kVals];
            Chunks<kTurn>::load(table + row.t * turns, item, pair_items, m);
            const float *a = gr[i], *b = gr[i] + kPairs;
            if (!any_outside) {
              // a cos - b sin', b cos + a sin' with sin' = -sin (the inverse turn)
              float na[kPairs];
              mul_each<kPairs>(o, a, m);
              mul_each<kPairs>(o + kPairs, b, m);
#pragma unroll
              for (int j = 0; j < kPairs; ++j) na[j] = -b[j];
              fma_each<kPairs>(o, na, m + kPairs, o);
              fma_each<kPairs>(o + kPairs, a, m + kPairs, o + kPairs);
            } else {
#pragma unroll
              for (int j = 0; j < kPairs; ++j) {
                o[j] = a[j], o[kPairs + j] = b[j];
                if (alone(item, j)) continue;
                o[j] = a[j] * m[j] - b[j] * m[kPairs + j];
                o[kPairs + j] = b[j] * m[j] + a[j] * m[kPairs + j];
              }
            }
#pragma unroll
            for (int j = 0; j < kVals; ++j) gr[i][j] = o[j];
          }
          float wi[kVals], sum[kPairs];
          Chunks<kVals>::load(w, item, p.items, wi);
          fma_each<kVals>(dw[i], gr[i], f[i], dw[i]);
          mul_each<kVals>(gr[i], gr[i], wi);
          mul_each<kPairs>(sum, gr[i], f[i]);
          fma_each<kPairs>(sum, gr[i] + kPairs, f[i] + kPairs, sum);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) along += sum[j];
        }
        along = head_sum(along, p.lanes, at, lane - at) * p.inv_dim;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int item = at + i * p.lanes;
          if (!on || item >= p.items) break;
          fma_all<kVals>(gr[i], f[i], -along, gr[i]);
          mul_all<kVals>(gr[i], gr[i], root);
          It::store(row.y, item, pair_items, p.half, gr[i]);
        }
      }
    };
    int slot = 0;
    for (int r0 = warp * in_warp; r0 < rows; r0 += groups) {
      Row row;
      if constexpr (kSlots > 0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots > 0 ? kSlots - 2 : 0) : "memory");
        take(c, slot, row);
        advance(c);
        // into the slot that the last row was worked on from
        ask(ahead, slot == 0 ? kSlots - 1 : slot - 1);
        if (++slot == kSlots) slot = 0;
      } else {
        row = next;
        load(ahead, next);
      }
      advance(ahead);
      work(row);
    }
    if constexpr (kSlots > 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (BACK) __syncthreads();  // the table is refilled
  }

  if constexpr (BACK) {
    if (!p.partial) return;
    // the warps' sums, then the CTA's
    __syncthreads();
    float* sums = table;  // kWarps rows of items * kVals
    const int width = p.items * kVals;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int item = at + i * p.lanes;
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        float s = dw[i][j];
        for (int q = 1; q < in_warp; ++q) {
          const float o = __shfl_sync(0xFFFFFFFFu, dw[i][j], (lane + q * p.lanes) & 31);
          if (sub == 0) s += o;
        }
        if (sub == 0 && item < p.items) sums[warp * width + item * kVals + j] = s;
      }
    }
    __syncthreads();
    for (int i = (int)threadIdx.x; i < width; i += kThreads) {
      const int item = i / kVals;
      const int e = place_of<NEIGH, V>(item, i - item * kVals, pair_items, p.half, p.dim);
      if (e < 0) continue;
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += sums[k * width + i];
      p.partial[(int64_t)blockIdx.x * p.dim + e] = s;
    }
  }
}

cudaError_t launch_as(const void* kernel, unsigned grid, unsigned threads, size_t smem, void** args,
                      cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// The lanes of a head, and the items of a lane: as few lanes idle as can be (of a warp, and of
// the last of a lane's items).
struct Split {
  int lanes, per_lane;
};
template <int V, bool BACK>
Split split_of(int items) {
  Split best{0, 0};
  double most = -1.0;
  // (a head of 512 values has at most 64 items of 8 values, 128 of 4, 512 of one)
  constexpr int kChoices[3] = {V == 1 ? 4 : 1, V == 1 ? 16 : 2, V == 1 ? 16 : V == 4 ? 4 : 2};
  for (int i : kChoices) {
    const int lanes = (items + i - 1) / i;
    if (lanes > 32) continue;
    const double used = (double)items / (lanes * i) * (32 / lanes * lanes) / 32;
    // (forwards two accesses of 8 values rather than one, where none idles: the steps of a walk
    // over more values, 8192 x 72 x 128 58 us against 62; backwards that takes too many registers)
    if (used > most + 0.1 || (!BACK && V == 8 && i == 2 && used >= most)) most = used, best = {lanes, i};
  }
  return best;
}

template <typename T, bool NEIGH, int V, bool BACK>
cudaError_t launch(HeadsParams& p, int sms, cudaStream_t stream) {
  p.items = p.half / Item<T, NEIGH, V>::kPairs + (p.dim - 2 * p.half) / V;
  const Split split = split_of<V, BACK>(p.items);
  p.lanes = split.lanes;
  const int groups = 32 / p.lanes * kWarps;
  using L = HeadsLayout<NEIGH, V, BACK>;
  const int pair_items = p.half / L::kPairs;
  const size_t weights = (size_t)2 * L::weights(p.items, pair_items) * sizeof(float);
  const size_t per_token = (size_t)L::turns(pair_items) * sizeof(float) + p.half;
  const int64_t most_tokens = std::max<int64_t>(1, std::min<int64_t>(BACK ? 32 : 8, (int64_t)((40960 - weights) / per_token)));
  size_t ring = 0;
  if constexpr (V > 1) {
    const int bytes = split.per_lane == 1   ? ring_bytes<T, NEIGH, V, 1, BACK>()
                      : split.per_lane == 2 ? ring_bytes<T, NEIGH, V, 2, BACK>()
                                            : ring_bytes<T, NEIGH, V, 4, BACK>();
    ring = (size_t)kThreads * bytes;
  }
  const void* kernel;
  unsigned grid;
  size_t smem;
  if (!BACK) {
    // as rotary_kernel.cu: as many tokens per CTA as give every lane three runs of heads, as long
    // as every SM has two CTAs; with fewer tokens shares of one token's heads
    const int64_t want = (int64_t)9 * groups;
    const int64_t spread = ((int64_t)p.tokens * p.heads + 2 * sms - 1) / (2 * sms);
    const int64_t per_cta = std::max<int64_t>(groups, std::min(want, spread));
    p.tile_tokens = (int32_t)std::min<int64_t>(most_tokens, std::max<int64_t>(1, per_cta / p.heads));
    p.shares = (int32_t)((p.heads + per_cta - 1) / per_cta);
    p.share_heads = (p.heads + p.shares - 1) / p.shares;
    p.shares = (p.heads + p.share_heads - 1) / p.share_heads;
    grid = (unsigned)(((int64_t)p.tokens + p.tile_tokens - 1) / p.tile_tokens * p.shares);
    smem = weights + p.tile_tokens * per_token;
  } else {
    // Tiles of the same number of tokens for each of a kind's CTAs, as few as shared memory allows
    // beside a second CTA (tiles that gave every lane six heads left half of the CTAs idle in the
    // end: 4099 x (12 + 4) x 80 fp32 25.3 us, 22.1 so), and as many CTAs for either kind of heads as
    // let both end together: in steps of the walk over rows, a tile's start costs about two, and
    // two more for every kBatch pairs of a thread.  (CTAs in proportion to the heads, where the few
    // key heads' tiles come last: 8192 x (64 + 8) x 128 bf16 127 us, 102 so.)
    const int key_heads = p.heads - p.query_heads;
    const int64_t ctas = heads_back_ctas(sms);
    const int64_t room = 227 * 1024 / heads_per_sm(split.per_lane, true) - 1024 - (int64_t)(ring + weights);
    const int64_t most = std::min(most_tokens, std::max<int64_t>(1, room / (int64_t)per_token));
    struct Walk {
      int64_t tile, cost;
    };
    auto walk_of = [&](int heads, int64_t among) {
      const int64_t even = std::max<int64_t>(1, (p.tokens + among - 1) / among);
      const int64_t rounds = (even + most - 1) / most, tile = (even + rounds - 1) / rounds;
      return Walk{tile, rounds * ((tile * heads + groups - 1) / groups + 2 + 2 * ((tile * p.half + 4 * kThreads - 1) / (4 * kThreads)))};
    };
    int64_t q = p.query_heads == 0 ? 0 : ctas;
    if (p.query_heads > 0 && key_heads > 0) {
      int64_t low = 1, high = ctas - 1;  // the fewest CTAs that end the query heads no later
      while (low < high) {
        const int64_t mid = (low + high) / 2;
        if (walk_of(p.query_heads, mid).cost > walk_of(key_heads, ctas - mid).cost) low = mid + 1;
        else high = mid;
      }
      q = low;
    }
    p.tile_tokens = q == 0 ? 1 : (int32_t)walk_of(p.query_heads, q).tile;
    p.key_tile_tokens = q == ctas ? 1 : (int32_t)walk_of(key_heads, ctas - q).tile;
    p.query_ctas = (int32_t)std::min<int64_t>(q, (p.tokens + p.tile_tokens - 1) / p.tile_tokens);
    grid = (unsigned)(p.query_ctas + std::min<int64_t>(ctas - q, (p.tokens + p.key_tile_tokens - 1) / p.key_tile_tokens));
    p.ctas = (int32_t)grid;
    smem = std::max(weights + std::max(p.tile_tokens, p.key_tile_tokens) * per_token, (size_t)kWarps * p.items * L::kVals * sizeof(float));
  }
  if constexpr (V == 1) {
    kernel = split.per_lane == 4 ? reinterpret_cast<const void*>(heads_kernel<T, NEIGH, V, 4, BACK>)
                                 : reinterpret_cast<const void*>(heads_kernel<T, NEIGH, V, 16, BACK>);
  } else {
    kernel = split.per_lane == 1 ? reinterpret_cast<const void*>(heads_kernel<T, NEIGH, V, 1, BACK>)
                                 : reinterpret_cast<const void*>(heads_kernel<T, NEIGH, V, 2, BACK>);
    if constexpr (V == 4)
      if (split.per_lane == 4) kernel = reinterpret_cast<const void*>(heads_kernel<T, NEIGH, V, 4, BACK>);
  }
  smem += ring;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  void* args[] = {&p};
  return launch_as(kernel, grid, kThreads, smem, args, stream);
}

template <typename T, bool BACK>
cudaError_t by_layout(HeadsParams& p, bool neighbours, int vec, int sms, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2)
    if (vec == 8)
      return neighbours ? launch<T, true, 8, BACK>(p, sms, stream) : launch<T, false, 8, BACK>(p, sms, stream);
  if (vec == 4)
    return neighbours ? launch<T, true, 4, BACK>(p, sms, stream) : launch<T, false, 4, BACK>(p, sms, stream);
  return neighbours ? launch<T, true, 1, BACK>(p, sms, stream) : launch<T, false, 1, BACK>(p, sms, stream);
}

template <bool BACK>
cudaError_t by_type(HeadsParams& p, int elem, bool neighbours, int vec, int sms, cudaStream_t stream) {
  switch (elem) {
    case kElemF16: return by_layout<__half, BACK>(p, neighbours, vec, sms, stream);
    case kElemBF16: return by_layout<__nv_bfloat16, BACK>(p, neighbours, vec, sms, stream);
    case kElemF32: return by_layout<float, BACK>(p, neighbours, vec, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace gb300

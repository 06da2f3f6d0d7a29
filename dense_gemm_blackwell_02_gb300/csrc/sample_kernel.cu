// The choice of the next token: for every row of logits z, with m the largest, T the temperature
// and w = exp((z - m) / T),
//     top-k     of the tokens in the order of their logits (equal ones in that of their index) the
//               first k stay
//     top-p     of those, the first until their w reach p of their sum
//     min-p     of those, the ones with w >= min_p
// and of what is left, in the order of the index, the first token whose running sum of w exceeds
// u times the whole, u a given random number.  T <= 0: the first of the largest logits.
//
// The answer is a whole number that hangs on borders: 10^5 of them in a row without limits, so
// that weights and sums good to 2^-24 would give another token than the formula in one row of a
// hundred.  A weight is therefore a pair of binary32 values (Weight), good to 2^-34 of itself,
// and sums are such pairs in a lane and whole numbers across lanes, whose additions' order does not
// matter: of 2^-42 in 64 bits, which hold 2^20 weights of 1, where short weights are enough, else of
// 2^-62 in 128 bits.  (Binary64 has 1/64 of binary32's rate on this GPU: sums over lanes in it took 25
// us of one row's 30.)  Weights below 2^-60 are 0; all others count: at the ends of u's range, which
// no short weight decides, the answer may be any of them.
//
// One read of the logits: bound by HBM, if the passes over them stay on chip.  A row belongs to
// a cluster of CTAs, each of which keeps its slice in shared memory, where it fits (else the later
// passes read L2), and finds the largest logit while the slice arrives.  Weights that good cost 60
// instructions, so they are computed for few:
//   - limits: a threshold that about 1400 of the row's logits reach (their number hardly depends on
//     the row: the q-th largest of the 32 lanes' largest logits, the middle one over all warps)
//     selects candidates for the cluster's first CTA, which sorts them by counting, cuts and draws
//     (short_list).  Top-p needs the whole row's sum too, from weights of 15 instructions, good to
//     2^-21 with their sums: enough unless the cut hangs on it.
//   - a nucleus, or top-k, of more than that (wide_row): the logits are counted by their distance
//     from the largest, which brackets the last token that stays by counts and estimated masses;
//     the bracket's tokens, a few hundred, are sorted, and the short weights' sum before it tells
//     which of them is the last.
//   - the draw among many (rough_draw): the same short weights' sums per warp, and the warp where u
//     falls walked through once more, unless the token hangs on them; then by whole weights
//     (exact_draw).
// What that leaves (top-p of a large top-k, a bracket of more than 2048 tokens, a border nearer
// than the short weights' error) takes the full way (exact_row): limits count the row's logits by
// their distance from the largest (2048 bins, 32 per power of two of the weight), which brackets
// the last token that stays: top-k's bin is known then, top-p's up to the weights' spread within a
// bin.  What lies in the bracket is gathered and sorted; too many for that are counted a second
// time in finer bins, and what then still is too many (equal logits) is bisected by value and cut
// by index.  All passes of it add up whole weights.
//
// Measured: one row of 128256 bf16 10 us without limits, 15 with top-k 50, 40 with top-p 0.9 or
// 0.99 of a flat row: the latency of its passes and of the cluster's barriers between them, about
// 1.5 us each.
// 256 rows of 128256 fp32 (19 us at HBM's rate): 57 us greedy, 87 to 93 without limits, 81 with top-k
// 50, 266 with top-p 0.9, 130 with mixed limits, 676 with top-p 0.9 after top-k 20000: three to four rounds of 72 rows, each of which
// waits for its own passes; memory is read ahead for the next round.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr float kPerLog2 = 32.0f;    // bins per power of two, first count
constexpr float kMostLog2 = 60.0f;   // weights below 2^-this are 0
constexpr int kWideBins = 1024;    // of the short way
constexpr int kList = 2048;          // candidates that are sorted
constexpr int kTable = 64;           // 2^(-j / 64)
constexpr int kMaxCluster = 8;
constexpr int kMostOrdered = 4096;   // rows
constexpr int kCopies = 8;           // of the table, for lanes side by side: fewer bank conflicts
constexpr uint32_t kTableBytes = kTable * kCopies * 2 * 4;
constexpr uint32_t kRegionBytes = kList * 8;  // two counts of kBins, or the candidates
static_assert(kRegionBytes == 2 * kBins * 4, "one region for both");
constexpr uint32_t kFixedSmem = kTableBytes + 2 * kRegionBytes;

template <typename V>
__device__ __forceinline__ V* cluster_at(V* p, uint32_t rank) {
  V* r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return r;
}

// (the barrier wants whole warps)
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  cluster_sync();
}

// A value as an unsigned number of the same order.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// NaN is never chosen; -0 is 0.
__device__ __forceinline__ float clean(float z) { return isnan(z) ? -__builtin_huge_valf() : z + 0.0f; }

// Sums of weights as whole numbers.  Fixed: in units of 2^-kFixedBits, of all of a row's weights,
// where a border that is not next to the sum decides; 2048 weights fit units of 2^-kListBits.  Whole:
// in units of 2^-kWholeBits, in which no weight that counts (2^-60 and more) is 0, so that a sum above
// 0 always has a token in it.
using Fixed = uint64_t;
constexpr int kFixedBits = 42, kListBits = 52, kWholeBits = 62;
using Whole = unsigned __int128;

// hi + lo, lo below half a step of hi.
struct Weight {
  float hi, lo;
  template <int BITS = kFixedBits>
  __device__ __forceinline__ Fixed fixed() const {
    constexpr float kUnit = (float)(1ull << BITS);
    return (Fixed)(__float2ll_rn(hi * kUnit) + __float2ll_rn(lo * kUnit));
  }
  // (a weight is at most 1 ...
  __device__ __forceinline__ Whole whole() const { return fixed<kWholeBits>(); }
  // ... a sum of them, any number)
  __device__ __forceinline__ Whole whole_sum() const {
    const float of = floorf(hi);
    return ((Whole)(uint64_t)of << kWholeBits) + (Whole)(__int128)(int64_t)Weight{hi - of, lo}.fixed<kWholeBits>();
  }
};

// x times a share in [0, 1), rounded down or up.
__device__ __forceinline__ Fixed share_of(Fixed x, float share, bool up) {
  const uint64_t f = (uint64_t)__float2ll_rz(share * 9223372036854775808.0f);  // 2^63, exact
  const uint64_t low = x * f;
  return (__umul64hi(x, f) << 1 | low >> 63) + (up && (low << 1) != 0 ? 1 : 0);
}
__device__ __forceinline__ Whole share_of(Whole x, float share, bool up) {
  const uint64_t f = (uint64_t)__float2ll_rz(share * 9223372036854775808.0f);
  const Whole high = (Whole)(uint64_t)(x >> 64) * f, low = (Whole)(uint64_t)x * f;  // (x below 2^83)
  return (high << 1) + (low >> 63) + (up && (uint64_t)(low << 65 >> 64) != 0 ? 1 : 0);
}
// In the other units.
__device__ __forceinline__ Fixed to_fixed(Whole x) { return (Fixed)(x >> (kWholeBits - kFixedBits)); }
__device__ __forceinline__ float to_float(Fixed x) { return __ull2float_rn(x) * (1.0f / (float)(1ull << kFixedBits)); }

struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(const Weight& w) {
    const float s = hi + w.hi, b = s - hi;
    lo += ((hi - (s - b)) + (w.hi - b)) + w.lo;
    hi = s;
  }
  __device__ __forceinline__ Fixed value() const { return Weight{hi, lo}.fixed(); }
  __device__ __forceinline__ Whole whole() const { return Weight{hi, lo}.whole_sum(); }
};

// A row's rules and a lane's way to the weights.
struct RowState {
  float m;          // the largest logit
  float scale_hi, scale_lo;  // log2(e) / T
  float cut_z;      // the last token that stays: logits above it, and equal ones up to its index
  int32_t cut_v;
  float min_p;
  const float* table;  // this lane's copy: entry j at 2 kCopies j words, hi then lo

  // -log2 of the weight, good to a few roundings: the same value for the same logit
  __device__ __forceinline__ float distance(float z) const { return z == m ? 0.0f : (m - z) * scale_hi; }
  __device__ __forceinline__ bool inside(float z, int32_t v) const {
    return z > cut_z || (z == cut_z && v <= cut_v);
  }
  __device__ __forceinline__ Weight weight(float z) const {
    // m - z and its rounding error (the exact error of a sum, whichever is larger), then both
    // times log2(e) / T
    const float d = m - z, b = d - m;
    const float dl = (m - (d - b)) + (-z - b);
    float t = d * scale_hi;
    float tl = fmaf(dl, scale_hi, fmaf(d, scale_lo, fmaf(d, scale_hi, -t)));
    if (z == m) t = 0.0f, tl = 0.0f;  // (also of infinities)
    // t = j / 64 + r, |r| <= 2^-7
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: the sum's last bits are round(64 t)
    const float y = fmaf(t, (float)kTable, kMagic);
    const int32_t j = __float_as_int(y) - __float_as_int(kMagic);
    const float r = fmaf(y - kMagic, -1.0f / kTable, t);
    // 2^-(r + tl) = 1 + x + (rest), x = -r ln 2 to 24 bits, the rest below 2^-15
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236017e-9f;
    const float x = -r * kLn2Hi;
    const float xl = fmaf(tl, -kLn2Hi, fmaf(r, -kLn2Lo, fmaf(r, -kLn2Hi, -x)));
    const float q = fmaf(fmaf(x, 1.0f / 24.0f, 1.0f / 6.0f), x, 0.5f);
    const float rest = fmaf(q * x, x, fmaf(xl, x, xl));
    const float* e = table + (j & (kTable - 1)) * 2 * kCopies;
    const float th = e[0], tlo = e[kCopies];
    const float p = th * x;
    const float pl = fmaf(th, rest, fmaf(th, x, -p)) + fmaf(tlo, x, tlo);
    const float w = th + p;
    const float wl = ((th - w) + p) + pl;
    const bool ok = t <= kMostLog2;  // (false for NaN: an infinite distance times 0)
    const float s = ok ? __int_as_float((127 - (j >> 6)) << 23) : 0.0f;
    return ok ? Weight{w * s, wl * s} : Weight{0.0f, 0.0f};
  }
  // The short weight: within exp2's two steps and a rounding of it, 2^-22 + 2^-24; with three
  // more roundings of a sum of eight, 2^-21.  (Not for infinite m or scale.)
  __device__ __forceinline__ float rough(float z) const {
    const float d = m - z, b = d - m;
    const float dl = (m - (d - b)) + (-z - b);
    const float t = d * scale_hi;
    const float tl = fmaf(dl, scale_hi, fmaf(d, scale_lo, fmaf(d, scale_hi, -t)));
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(-t));
    w = fmaf(w * tl, -0.693147182464599609375f, w);
    return t <= kMostLog2 ? w : 0.0f;
  }
  // ... 0 below min_p; `near`: too near it to say.
  __device__ __forceinline__ float rough_kept(float z, bool& near) const {
    const float w = rough(z);
    near |= min_p > 0.0f && fabsf(w - min_p) <= 0x1p-20f * min_p && z != m;
    return w >= min_p ? w : 0.0f;
  }
  // The weight of a token that stays, 0 of the others.
  __device__ __forceinline__ Weight kept(float z, int32_t v) const {
    if (!inside(z, v)) return {0.0f, 0.0f};
    const Weight w = weight(z);
    return w.hi > min_p || (w.hi == min_p && w.lo >= 0.0f) ? w : Weight{0.0f, 0.0f};
  }
};

// Where the last token that stays is looked for: first-count bins lo..hi, within them bins
// lo2..hi2 of a second count that starts at `from` with `per` bins per power of two.
struct Bracket {
  int32_t lo, hi, lo2, hi2;
  float from, per;   // (per 0: no second count yet)
  uint32_t before;   // tokens before it
  uint32_t count;    // tokens in it
  uint32_t all;      // tokens counted
  static __device__ __forceinline__ Bracket everything() {
    return {0, kBins - 1, 0, kBins - 1, 0.0f, 0.0f, 0u, 0u, 0u};
  }
  __device__ __forceinline__ int fine(float t) const { return min(max((int)((t - from) * per), 0), kBins - 1); }
  // -1: before the bracket, 0: in it, 1: behind it
  __device__ __forceinline__ int place(float t) const {
    const int b = (int)(t * kPerLog2);
    if (b < lo) return -1;
    if (b > hi) return 1;
    if (per == 0.0f) return 0;
    const int f = fine(t);
    return f < lo2 ? -1 : f > hi2 ? 1 : 0;
  }
};

struct Cut {
  float z;
  int32_t v;
};

// A row's limits, as the cluster's first CTA read them: what its CTAs do together must not differ,
// even where the vectors change meanwhile (which makes the row's answer anything, no more).
struct Rules {
  float scale_hi, scale_lo;  // log2(e) / temperature
  int32_t greedy, top_k;
  float top_p, min_p;
};

struct Shared {
  Fixed slots[2][kMaxCluster];      // a sum from every CTA of the cluster, in turn
  Fixed more_slots[kMaxCluster];
  Fixed parts[kWarps];
  Whole whole_slots[2][kMaxCluster];
  Whole whole_parts[kWarps];
  uint32_t count_parts[kWarps];
  float low_parts[kWarps], high_parts[kWarps];
  uint32_t ends[2];
  float best[kMaxCluster], quantile[kMaxCluster];
  uint32_t counts[kMaxCluster];
  int32_t first[kMaxCluster];
  float warp_best[kWarps], warp_quantile[kWarps];
  Bracket bracket;
  Cut cut;
  uint32_t listed, mine, base;
  Fixed warp_sums[kWarps];          // of what stays
  int32_t found, found_hi, found_lo, last;
  int32_t unsure, near_draw;        // the cut, or the draw, hangs on the short weights' errors
  Rules own_rules, rules;
};

// A CTA's part of a row: tokens v0..v0+n-1; position i is token v0 + i - shift, so that vectors of
// positions are aligned in memory.  A warp owns vectors q0..q1-1, a lane every 32nd of them.
template <typename T>
struct Part {
  static constexpr int V = 16 / (int)sizeof(T);  // logits per access
  const T* in;
  T* slice;
  int32_t v0, n, shift, vectors, q0, q1;
  int32_t row;
  bool resident;

  __device__ __forceinline__ int32_t first_of(int warp) const {
    return (int32_t)((int64_t)warp * vectors / kWarps);
  }
  __device__ __forceinline__ Pack<T, V> from_memory(int32_t q) const {
    Pack<T, V> x;
    if (q * V >= shift && q * V - shift + V <= n) {
      x = *reinterpret_cast<const Pack<T, V>*>(in + q * V - shift);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int32_t i = q * V + j - shift;
        x.v[j] = i >= 0 && i < n ? in[i] : from_f32<T>(-__builtin_huge_valf());
      }
    }
    return x;
  }
  __device__ __forceinline__ Pack<T, V> packed(int32_t q) const {
    return resident ? *reinterpret_cast<const Pack<T, V>*>(slice + q * V) : from_memory(q);
  }
  __device__ __forceinline__ void vector(int32_t q, float (&z)[V]) const { unpack(packed(q), z); }
  // The token of a vector's first logit.
  __device__ __forceinline__ int32_t token(int32_t q) const { return v0 + q * V - shift; }
  // f(logit, token) for this lane's share of the warp's
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    vectors_of([&](const float (&z)[V], int32_t q) {
#pragma unroll
      for (int j = 0; j < V; ++j) f(clean(z[j]), token(q) + j);
    });
  }
  // f(logits, vector) likewise, the next vector on its way meanwhile if it comes from L2, as those of
  // long binary32 rows do (256 x 128256, top-k 50 86 -> 81 us; 16 bits, in shared memory, 94 -> 97)
  template <typename F>
  __device__ __forceinline__ void vectors_of(F f) const {
    int32_t q = q0 + (int)lane_id();
    float z[V];
    if constexpr (sizeof(T) == 4) {
      if (q >= q1) return;
      Pack<T, V> x = packed(q);
      for (; q < q1; q += 32) {
        unpack(x, z);
        if (q + 32 < q1) x = packed(q + 32);
        f(z, q);
      }
    } else {
      for (; q < q1; q += 32) {
        vector(q, z);
        f(z, q);
      }
    }
  }
};

// The larger of two, element by element; NaN loses.
__device__ __forceinline__ float largest(const Pack<float, 4>& x) {
  return fmaxf(fmaxf(x.v[0], x.v[1]), fmaxf(x.v[2], x.v[3]));
}
template <typename T>
__device__ __forceinline__ float largest(const Pack<T, 8>& x) {
  using P = typename PairOf<T>::type;
  const P* w = reinterpret_cast<const P*>(&x);
  const float2 f = pair_f32(__hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
  return fmaxf(f.x, f.y);
}

// ----------------------------------------------------------------- sums over threads --
template <typename S>
__device__ __forceinline__ S from_lane_xor(S s, int off) { return __shfl_xor_sync(0xFFFFFFFFu, s, off); }
__device__ __forceinline__ Whole from_lane_xor(Whole s, int off) {
  return (Whole)__shfl_xor_sync(0xFFFFFFFFu, (uint64_t)(s >> 64), off) << 64 |
         __shfl_xor_sync(0xFFFFFFFFu, (uint64_t)s, off);
}
template <typename S>
__device__ __forceinline__ S from_lane_up(S s, int off) { return __shfl_up_sync(0xFFFFFFFFu, s, off); }
__device__ __forceinline__ Whole from_lane_up(Whole s, int off) {
  return (Whole)__shfl_up_sync(0xFFFFFFFFu, (uint64_t)(s >> 64), off) << 64 |
         __shfl_up_sync(0xFFFFFFFFu, (uint64_t)s, off);
}
// Of all threads, in every thread, over parts[kWarps].
template <typename S>
__device__ __forceinline__ S block_sum(S s, S* parts) {
  const int warp = (int)warp_id();
  for (int off = 16; off > 0; off >>= 1) s += from_lane_xor(s, off);
  __syncthreads();
  if (lane_id() == 0) parts[warp] = s;
  __syncthreads();
  S all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += parts[w];
  return all;
}
__device__ __forceinline__ Fixed block_sum(Fixed s, Shared& sh) { return block_sum(s, sh.parts); }
// Of the threads up to and with this one, over parts[kWarps].
template <typename S>
__device__ __forceinline__ S block_scan(S s, S* parts) {
  const int warp = (int)warp_id(), lane = (int)lane_id();
  for (int off = 1; off < 32; off <<= 1) {
    const S o = from_lane_up(s, off);
    if (lane >= off) s += o;
  }
  __syncthreads();
  if (lane == 31) parts[warp] = s;
  __syncthreads();
  S before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) before += w < warp ? parts[w] : S(0);
  return before + s;
}

// Rows number `first` and `second` (p.rows and more: that) in the order in which they run: those
// that may take several times the others' time, top-p without top-k, before the others.
__device__ __forceinline__ int2 in_order(const SampleParams& p, int32_t first, int32_t second, Shared& sh) {
  const int tid = (int)threadIdx.x;
  auto long_row = [&](int32_t r) {
    const int32_t k = p.top_k ? p.top_k[r] : 0;
    return p.top_p[r] < 1.0f && !(k >= 1 && k < p.vocab) && (!p.temperature || p.temperature[r] > 0.0f);
  };
  const int32_t each = (p.rows + kThreads - 1) / kThreads, a = min(tid * each, p.rows), b = min(a + each, p.rows);
  uint32_t own = 0;
  for (int32_t r = a; r < b; ++r) own += long_row(r);
  if (tid == 0) sh.found_lo = first, sh.found_hi = second;
  int32_t at = (int32_t)(block_scan(own, sh.count_parts) - own), all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += (int32_t)sh.count_parts[w];
  int32_t other = all + a - at;
  for (int32_t r = a; r < b; ++r) {
    const int32_t place = long_row(r) ? at++ : other++;
    if (place == first) sh.found_lo = r;
    if (place == second) sh.found_hi = r;
  }
  __syncthreads();
  const int2 rows = make_int2(sh.found_lo, sh.found_hi);
  __syncthreads();
  return rows;
}

// The middle one of n values (the n / 2-th in descending order).
__device__ __forceinline__ float middle(const float* v, int n) {
  float m = v[0];
  for (int i = 0; i < n; ++i) {
    int above = 0;
    for (int j = 0; j < n; ++j) above += v[j] > v[i] || (v[j] == v[i] && j < i);
    if (above == n / 2) m = v[i];
  }
  return m;
}

// w / whole, rounded once.
__device__ __forceinline__ float quotient(const Weight& w, Fixed whole) {
  constexpr float kUnit = (float)(1ull << kFixedBits);
  const float wh = to_float(whole);
  const float wl = __ll2float_rn((int64_t)(whole - (Fixed)__float2ll_rn(wh * kUnit))) * (1.0f / kUnit);
  const float q = __fdiv_rn(w.hi, wh);
  return q + __fdiv_rn(fmaf(-q, wh, w.hi) + fmaf(-q, wl, w.lo), wh);
}

// The mass that top-p asks of a sum, rounded up, and the draw's share of it.
template <typename S>
__device__ __forceinline__ S top_of(S whole, float top_p) {
  return top_p > 0.0f ? share_of(whole, top_p, true) : (S)0;
}
template <typename S>
__device__ __forceinline__ S drawn_of(S whole, float u) {  // (u of 1 and more: the last)
  return u >= 1.0f ? whole : u > 0.0f ? share_of(whole, u, false) : (S)0;
}

// The first token, in the order of the index, at which the running sum of f exceeds goal_of(the
// whole); the last one with f > 0 where none does.  In the owner's threads only: `done` of
// (token, f there, whole).  `lane_sum`: f's sum over this lane's share.
template <typename T, typename G, typename F, typename D>
__device__ __forceinline__ void locate_in(const Part<T>& part, Shared& sh, int turn, uint32_t ctas, uint32_t rank,
                                          Whole lane_sum, G goal_of, F f, D done) {
  constexpr int V = Part<T>::V;
  const int tid = (int)threadIdx.x;
  const Whole mine = block_sum(lane_sum, sh.whole_parts);
  if (tid < (int)ctas) *cluster_at(&sh.whole_slots[turn][rank], (uint32_t)tid) = mine;
  cluster_barrier();
  Whole whole = 0;
  for (uint32_t c = 0; c < ctas; ++c) whole += sh.whole_slots[turn][c];
  const Whole goal = goal_of(whole);
  const bool past = goal >= whole;  // beyond all of it: the last token
  Whole before = 0, run = 0;
  int owner = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const Whole of = sh.whole_slots[turn][c];
    if (of > 0 && (past || run <= goal)) owner = (int)c, before = run;
    run += of;
  }
  if (owner != (int)rank) return;
  // the warp ...
  int w_at = 0;
  run = before;
  for (int w = 0; w < kWarps; ++w) {
    const Whole of = sh.whole_parts[w];
    if (of > 0 && (past || run <= goal)) w_at = w, before = run;
    run += of;
  }
  // ... whose vectors all threads now share, in runs
  const int32_t a = part.first_of(w_at), b = part.first_of(w_at + 1);
  const int32_t each_q = (b - a + kThreads - 1) / kThreads;
  const int32_t qa = a + tid * each_q, qb = min(qa + each_q, b);
  Whole own = 0;
  auto walk = [&](auto g) {
    for (int32_t q = qa; q < qb; ++q) {
      float z[V];
      part.vector(q, z);
#pragma unroll
      for (int j = 0; j < V; ++j) g(clean(z[j]), part.token(q) + j);
    }
  };
  walk([&](float z, int32_t v) { own += f(z, v).whole(); });
  if (tid == 0) sh.found = -1;
  run = before + block_scan(own, sh.whole_parts) - own;  // (has the barriers)
  // the last thread that begins at or below the goal and has something
  if (own > 0 && (past || run <= goal)) atomicMax(&sh.found, tid);
  __syncthreads();
  if (tid == sh.found) {
    int32_t token = -1;
    Weight wt{0.0f, 0.0f};
    walk([&](float z, int32_t v) {
      const Weight w = f(z, v);
      const Whole of = w.whole();
      if (of > 0 && (past || run <= goal)) token = v, wt = w;
      run += of;
    });
    done(token, wt, whole);
  }
}

// Two weights at a time, as RowState::weight computes them, operation by operation, with
// instructions that hold two values.  For finite m and scale; logits below `least` (further than
// kMostLog2 from m; NaN too) are taken as that, whose weight is 0.
using F2 = uint64_t;
__device__ __forceinline__ F2 two(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void parts_of(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
struct Weights2 {
  F2 hi, lo;
};
struct Sum2 {
  F2 hi = 0, lo = 0;
  __device__ __forceinline__ void add(const Weights2& w) {
    const F2 minus = two(-1.0f, -1.0f);
    const F2 s = add2(hi, w.hi), b = fma2(hi, minus, s);
    const F2 x = fma2(fma2(b, minus, s), minus, hi), y = fma2(b, minus, w.hi);
    lo = add2(lo, add2(add2(x, y), w.lo));
    hi = s;
  }
  __device__ __forceinline__ Fixed value() const {
    float a, b, c, d;
    parts_of(hi, a, b);
    parts_of(lo, c, d);
    return Weight{a, c}.fixed() + Weight{b, d}.fixed();
  }
  __device__ __forceinline__ Whole whole() const {
    float a, b, c, d;
    parts_of(hi, a, b);
    parts_of(lo, c, d);
    return Weight{a, c}.whole_sum() + Weight{b, d}.whole_sum();
  }
};
struct Pairs {
  F2 m, scale, minus_scale, scale_lo;
  float least;
  const float* table;
  bool usable;
  __device__ __forceinline__ explicit Pairs(const RowState& st)
      : m(two(st.m, st.m)),
        scale(two(st.scale_hi, st.scale_hi)),
        minus_scale(two(-st.scale_hi, -st.scale_hi)),
        scale_lo(two(st.scale_lo, st.scale_lo)),
        least(st.m - 61.0f / st.scale_hi),
        table(st.table) {
    // (`least` has to lie where it says: next to an m of 10^9 there are no such values)
    usable = isfinite(st.m) && isfinite(st.scale_hi) && least > -1e37f && (st.m - least) * st.scale_hi > 60.5f;
  }
  __device__ __forceinline__ Weights2 weights(float z0, float z1, bool keep0, bool keep1) const {
    const F2 minus = two(-1.0f, -1.0f);
    const F2 z = two(fmaxf(z0, least), fmaxf(z1, least));
    const F2 d = fma2(z, minus, m), nb = fma2(d, minus, m);
    const F2 dl = add2(fma2(add2(d, nb), minus, m), fma2(z, minus, nb));
    const F2 nt = mul2(d, minus_scale);
    const F2 tl = fma2(dl, scale, fma2(d, scale_lo, fma2(d, scale, nt)));
    constexpr float kMagic = 12582912.0f;
    const F2 y = fma2(nt, two(-(float)kTable, -(float)kTable), two(kMagic, kMagic));
    float y0, y1, t0, t1;
    parts_of(y, y0, y1);
    parts_of(nt, t0, t1);
    const int32_t j0 = __float_as_int(y0) - __float_as_int(kMagic), j1 = __float_as_int(y1) - __float_as_int(kMagic);
    const F2 nr = fma2(add2(y, two(-kMagic, -kMagic)), two(1.0f / kTable, 1.0f / kTable), nt);
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236017e-9f;
    const F2 ln2 = two(kLn2Hi, kLn2Hi), minus_ln2 = two(-kLn2Hi, -kLn2Hi);
    const F2 x = mul2(nr, ln2), nx = mul2(nr, minus_ln2);
    const F2 xl = fma2(tl, minus_ln2, fma2(nr, two(kLn2Lo, kLn2Lo), fma2(nr, ln2, nx)));
    const F2 q = fma2(fma2(x, two(1.0f / 24.0f, 1.0f / 24.0f), two(1.0f / 6.0f, 1.0f / 6.0f)), x, two(0.5f, 0.5f));
    const F2 rest = fma2(mul2(q, x), x, fma2(xl, x, xl));
    const float* e0 = table + (j0 & (kTable - 1)) * 2 * kCopies;
    const float* e1 = table + (j1 & (kTable - 1)) * 2 * kCopies;
    const F2 th = two(e0[0], e1[0]), tlo = two(e0[kCopies], e1[kCopies]);
    const F2 p = mul2(th, x);
    const F2 pl = add2(fma2(th, rest, fma2(th, x, mul2(th, nx))), fma2(tlo, x, tlo));
    const F2 w = add2(th, p);
    const F2 wl = add2(add2(fma2(w, minus, th), p), pl);
    const F2 s = two(keep0 && -t0 <= kMostLog2 ? __int_as_float((127 - (j0 >> 6)) << 23) : 0.0f,
                     keep1 && -t1 <= kMostLog2 ? __int_as_float((127 - (j1 >> 6)) << 23) : 0.0f);
    return {mul2(w, s), mul2(wl, s)};
  }
};

// What stays is known (st): the token by whole weights.  Every CTA of the cluster comes here, or
// none.
template <typename T>
__device__ __noinline__ void exact_draw(const SampleParams& p, const Part<T>& part, RowState st, Shared& sh, int turn) {
  constexpr int V = Part<T>::V;
  const int row = part.row;
  const Pairs pairs(st);
  Whole mine;
  if (pairs.usable) {
    Sum2 sum;
    for (int32_t q = part.q0 + (int)lane_id(); q < part.q1; q += 32) {
      float z[V];
      part.vector(q, z);
      const int32_t v = part.token(q);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const bool a = st.inside(z[j], v + j), b = st.inside(z[j + 1], v + j + 1);
        Weights2 w = pairs.weights(z[j], z[j + 1], a, b);
        if (st.min_p > 0.0f) {
          float a0, a1, b0, b1;
          parts_of(w.hi, a0, a1);
          parts_of(w.lo, b0, b1);
          const bool on0 = a0 > st.min_p || (a0 == st.min_p && b0 >= 0.0f);
          const bool on1 = a1 > st.min_p || (a1 == st.min_p && b1 >= 0.0f);
          w = {two(on0 ? a0 : 0.0f, on1 ? a1 : 0.0f), two(on0 ? b0 : 0.0f, on1 ? b1 : 0.0f)};
        }
        sum.add(w);
      }
    }
    mine = sum.whole();
  } else {
    Sum sum;
    part.each([&](float z, int32_t v) { sum.add(st.kept(z, v)); });
    mine = sum.whole();
  }
  const float u = p.random[row];
  locate_in<T>(part, sh, turn, (uint32_t)p.cluster, cluster_ctarank(), mine,
               [&](Whole whole) { return drawn_of(whole, u); },
               [&](float z, int32_t v) { return st.kept(z, v); },
               [&](int32_t token, Weight w, Whole whole) {
                 p.tokens[row] = token;
                 if (p.probs) p.probs[row] = quotient(w, to_fixed(whole));
               });
}

// The full way.  Every CTA of the cluster comes here, or none.
template <typename T>
__device__ __noinline__ void exact_row(const SampleParams& p, const Part<T>& part, RowState st, Shared& sh,
                                       uint32_t* region, int turn) {
  const int tid = (int)threadIdx.x;
  const uint32_t ctas = (uint32_t)p.cluster, rank = cluster_ctarank();
  const int32_t k = sh.rules.top_k;
  const float top_p = sh.rules.top_p;
  bool by_count = k >= 1 && k < p.vocab;
  const bool by_mass = top_p < 1.0f;
  auto cluster_sum = [&](Whole s) {  // of all CTAs' block sums, and a barrier of the cluster
    const Whole mine = block_sum(s, sh.whole_parts);
    if (tid < (int)ctas) *cluster_at(&sh.whole_slots[turn][rank], (uint32_t)tid) = mine;
    cluster_barrier();
    Whole all = 0;
    for (uint32_t c = 0; c < ctas; ++c) all += sh.whole_slots[turn][c];
    turn ^= 1;
    return all;
  };

  auto locate = [&](auto goal_of, auto f, auto done) {
    Sum lane_sum;
    part.each([&](float z, int32_t v) { lane_sum.add(f(z, v)); });
    locate_in<T>(part, sh, turn, ctas, rank, lane_sum.whole(), goal_of, f, done);
    turn ^= 1;
  };

  // Counts the tokens that stay so far, in the bracket's next bins; the cluster's first CTA
  // brackets the last token more closely: the one that makes the count reach `count_goal`, or, with
  // that 0, the mass reach `goal` (with `base` before the bracket).
  auto narrow = [&](Bracket br, uint32_t count_goal, Whole goal, Whole base) {
    uint32_t* counts = region;
    uint32_t* sums = region + kBins;
    for (int i = tid; i < kBins; i += kThreads) counts[i] = 0;
    __syncthreads();
    const bool second = br.per != 0.0f;
    part.each([&](float z, int32_t v) {
      const float t = st.distance(z);
      if (!(t <= kMostLog2) || !st.inside(z, v)) return;
      const int b = max((int)(t * kPerLog2), 0);
      if (!second) atomicAdd(counts + b, 1u);
      else if (b >= br.lo && b <= br.hi) atomicAdd(counts + br.fine(t), 1u);
    });
    cluster_barrier();
    const int per = kBins / (int)ctas;
    for (int i = tid; i < per; i += kThreads) {
      const int b = (int)rank * per + i;
      uint32_t s = 0;
      for (uint32_t c = 0; c < ctas; ++c) s += *cluster_at(counts + b, c);
      *cluster_at(sums + b, 0u) = s;
    }
    cluster_barrier();
    if (rank == 0) {
      constexpr int kMine = kBins / kThreads;
      uint32_t mine[kMine], c = 0;
      float lo = 0.0f, hi = 0.0f;
      // the weights of a bin's tokens, bracketed: with 2^-16 for the distances' roundings and those
      // of these sums
      constexpr float kDown = 1.0f - 0x1p-16f, kUp = 1.0f + 0x1p-16f;
      const float start = second ? br.from : 0.0f, width = second ? 1.0f / br.per : 1.0f / kPerLog2;
      auto bound = [&](int b) { return exp2f(-(start + (float)b * width)); };
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int b = tid * kMine + i;
        mine[i] = sums[b];
        c += mine[i];
        lo += (float)mine[i] * bound(b + 1);
        hi += (float)mine[i] * bound(b);
      }
      if (tid == 0) sh.found = sh.found_lo = sh.found_hi = kBins - 1;
      uint32_t run_c = block_scan(c, sh.count_parts) - c;
      const uint32_t before_c = run_c;
      if (count_goal) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          run_c += mine[i];
          if (run_c >= count_goal) atomicMin(&sh.found, tid * kMine + i);
        }
      } else {
        const float goal_f = to_float(to_fixed(goal)), base_f = to_float(to_fixed(base));
        float run_lo = base_f + (block_scan(lo, sh.low_parts) - lo), run_hi = base_f + (block_scan(hi, sh.high_parts) - hi);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int b = tid * kMine + i;
          run_lo += (float)mine[i] * bound(b + 1);
          run_hi += (float)mine[i] * bound(b);
          if (run_hi * kUp >= goal_f) atomicMin(&sh.found_lo, b);
          if (run_lo * kDown >= goal_f) atomicMin(&sh.found_hi, b);
        }
      }
      __syncthreads();
      const int from = count_goal ? sh.found : sh.found_lo, to = count_goal ? sh.found : sh.found_hi;
      // tokens before the bracket, and up to its end
      uint32_t r = before_c;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int b = tid * kMine + i;
        if (b == from) sh.ends[0] = r;
        r += mine[i];
        if (b == to) sh.ends[1] = r;
      }
      if (tid == kThreads - 1 && !second) br.all = r;
      __syncthreads();
      if (tid == kThreads - 1) {
        if (second) br.lo2 = from, br.hi2 = to;
        else br.lo = from, br.hi = to;
        br.before += sh.ends[0];
        br.count = sh.ends[1] - sh.ends[0];
        for (uint32_t cta = 0; cta < ctas; ++cta) *cluster_at(&sh.bracket, cta) = br;
        sh.listed = 0;
      }
    }
    cluster_barrier();
    return sh.bracket;
  };
  // The sum of the weights of what stays so far and lies before the bracket.
  auto mass_before = [&](const Bracket& br) {
    Sum s;
    part.each([&](float z, int32_t v) {
      const float t = st.distance(z);
      if (t <= kMostLog2 && br.place(t) < 0 && st.inside(z, v)) s.add(st.weight(z));
    });
    return cluster_sum(s.whole());
  };
  auto mass_of_all = [&] {
    Sum s;
    part.each([&](float z, int32_t v) {
      if (st.inside(z, v)) s.add(st.weight(z));
    });
    return cluster_sum(s.whole());
  };
  // The second count's bins over the first one's bracket.
  auto finer = [&](Bracket br) {
    br.from = (float)br.lo / kPerLog2;
    br.per = (float)kBins * kPerLog2 / (float)(br.hi - br.lo + 1);
    br.lo2 = 0, br.hi2 = kBins - 1;
    return br;
  };
  // The bracket's tokens, sorted by the first CTA, of which `pick`, in that CTA's threads, says
  // the place of the last that stays.
  auto sorted = [&](const Bracket& br, auto pick) {
    uint64_t* list = reinterpret_cast<uint64_t*>(region);
    uint64_t* far_list = cluster_at(list, 0u);
    uint32_t* far_count = cluster_at(&sh.listed, 0u);
    part.each([&](float z, int32_t v) {
      const float t = st.distance(z);
      if (!(t <= kMostLog2) || br.place(t) != 0 || !st.inside(z, v)) return;
      const uint32_t at = atomicAdd(far_count, 1u);
      if (at < kList) far_list[at] = (uint64_t)order_key(z) << 32 | (uint32_t)~v;
    });
    cluster_barrier();
    if (rank == 0) {
      const int count = (int)min(sh.listed, (uint32_t)kList);
      int size = 64;
      while (size < count) size *= 2;
      for (int i = count + tid; i < size; i += kThreads) list[i] = 0;
      __syncthreads();
      for (int len = 2; len <= size; len *= 2)
        for (int gap = len / 2; gap > 0; gap /= 2) {
          for (int i = tid; i < size / 2; i += kThreads) {
            const int a = 2 * i - (i & (gap - 1)), b = a + gap;
            const uint64_t x = list[a], y = list[b];
            if ((x < y) == ((a & len) == 0)) list[a] = y, list[b] = x;
          }
          __syncthreads();
        }
      pick(list, count);
      __syncthreads();
      if (tid == 0) {
        const uint64_t c = list[max(min(sh.found, count - 1), 0)];
        const Cut cut{key_value((uint32_t)(c >> 32)), (int32_t)~(uint32_t)c};
        for (uint32_t cta = 0; cta < ctas; ++cta) *cluster_at(&sh.cut, cta) = cut;
      }
    }
    cluster_barrier();
    st.cut_z = sh.cut.z;
    st.cut_v = sh.cut.v;
  };
  auto listed_weight = [&](const uint64_t* list, int i) { return st.weight(key_value((uint32_t)(list[i] >> 32))); };
  // In the first CTA: the first place of list[0..count) at which the running mass reaches `goal`,
  // or (share) that part of the list's mass.
  auto place_of_mass = [&](const uint64_t* list, int count, Whole base, auto goal_of) {
    constexpr int kMine = kList / kThreads;
    Whole w[kMine], s = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int at = tid * kMine + i;
      w[i] = at < count ? st.weight(key_value((uint32_t)(list[at] >> 32))).whole() : 0;
      s += w[i];
    }
    const Whole goal = goal_of(block_sum(s, sh.whole_parts));
    if (tid == 0) sh.found = count - 1;
    Whole run = base + (block_scan(s, sh.whole_parts) - s);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      run += w[i];
      if (tid * kMine + i < count && run >= goal) atomicMin(&sh.found, tid * kMine + i);
    }
  };
  // Too many equal or nearly equal ones: the largest value of which the tokens at or above reach
  // the goal, by bisection, and then the index at which its equals do.
  auto bisected = [&](bool count_goal, Whole goal) {
    uint32_t lo = order_key(-3.402823466e38f), hi = order_key(st.m);
    auto above = [&](uint32_t key, bool equal) {
      const float edge = key_value(key);
      Sum s;
      part.each([&](float z, int32_t v) {
        if ((z > edge || (equal && z == edge)) && st.inside(z, v)) {
          const Weight w = st.weight(z);
          if (w.hi > 0.0f) s.add(count_goal ? Weight{1.0f, 0.0f} : w);
        }
      });
      return cluster_sum(s.whole());
    };
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      if (above(mid, true) >= goal) lo = mid;
      else hi = mid - 1;
    }
    const float edge = key_value(lo);
    const Whole before = above(lo, false), lack = goal > before ? goal - before : 0;
    const Whole one = count_goal ? (Whole)1 << kWholeBits : st.weight(edge).whole();
    uint32_t need = 1;  // the fewest of the equals that reach the goal: (lack / one, rounded up)
    for (uint32_t bit = (uint32_t)kMaxSampleVocab; bit > 0; bit /= 2)
      if ((need + bit - 1) * one < lack) need += bit;
    // the need-th of the equals, or their last
    const RowState so_far = st;
    locate([&](Whole) { return ((Whole)need << kWholeBits) - ((Whole)1 << (kWholeBits - 1)); },
           [&](float z, int32_t v) { return Weight{z == edge && so_far.inside(z, v) ? 1.0f : 0.0f, 0.0f}; },
           [&](int32_t token, Weight, Whole) {
             const Cut cut{edge, token};
             for (uint32_t cta = 0; cta < ctas; ++cta) *cluster_at(&sh.cut, cta) = cut;
           });
    cluster_barrier();
    st.cut_z = sh.cut.z;
    st.cut_v = sh.cut.v;
  };

  bool mass_done = false;
  if (by_count) {
    Bracket br = narrow(Bracket::everything(), (uint32_t)k, 0, 0);
    if ((uint32_t)k >= br.all) {
      by_count = false;
    } else if (br.before + br.count <= kList) {
      // all that stays fits the list: top-p is decided there too
      br.lo = 0, br.before = 0;
      sorted(br, [&](const uint64_t* list, int count) {
        const int kept = min(k, count);
        if (by_mass) place_of_mass(list, kept, 0, [&](Whole all) { return top_of(all, top_p); });
        else if (tid == 0) sh.found = kept - 1;
      });
      mass_done = true;
    } else {
      if (br.count > kList) br = narrow(finer(br), (uint32_t)k - br.before, 0, 0);
      if (br.count <= kList)
        sorted(br, [&](const uint64_t*, int) {
          if (tid == 0) sh.found = k - 1 - (int)br.before;
        });
      else
        bisected(true, (Whole)k << kWholeBits);
    }
  }
  if (by_mass && !mass_done) {
    const Whole goal = top_of(mass_of_all(), top_p);
    Bracket br = narrow(Bracket::everything(), 0, goal, 0);
    if (br.count > kList) {
      const Whole base = mass_before(br);
      br = narrow(finer(br), 0, goal, base);
    }
    if (br.count <= kList) {
      const Whole base = mass_before(br);
      sorted(br, [&](const uint64_t* list, int count) {
        place_of_mass(list, count, base, [&](Whole) { return goal; });
      });
    } else {
      bisected(false, goal);
    }
  }

  st.min_p = fminf(fmaxf(sh.rules.min_p, 0.0f), 1.0f);  // (fmaxf: NaN is 0)
  exact_draw<T>(p, part, st, sh, turn);
}

// The first CTA's candidates, at most kList in registers, `kMine` to a thread: e[j] is number tid +
// j * kThreads of n, its logit's order above, the complement of its index below.
struct Candidates {
  static constexpr int kMine = kList / kThreads;
  uint64_t e[kMine];
  int n;
  __device__ __forceinline__ Candidates(const uint64_t* list, int n_) : n(n_) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) e[j] = has(j) ? list[(int)threadIdx.x + j * kThreads] : 0;
  }
  __device__ __forceinline__ bool has(int j) const { return (int)threadIdx.x + j * kThreads < n; }
  __device__ __forceinline__ float logit(int j) const { return key_value((uint32_t)(e[j] >> 32)); }
  __device__ __forceinline__ int32_t token(int j) const { return (int32_t)~(uint32_t)e[j]; }
  // Every candidate's rank: counted into bins, laid out bin by bin, and compared with its bin's;
  // bin_of(j) of kBins, and key_of(j), of which the larger comes first.  `placed` and `bins` are
  // kRegionBytes each.
  template <typename B, typename F>
  __device__ __forceinline__ void ranks(Shared& sh, void* placed_, uint32_t* bins, B bin_of, F key_of,
                                        int (&rank)[kMine]) const {
    using K = decltype(key_of(0));
    K* placed = static_cast<K*>(placed_);
    const int tid = (int)threadIdx.x;
    for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    int bin[kMine], at[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      bin[j] = has(j) ? bin_of(j) : 0;
      at[j] = has(j) ? (int)atomicAdd(bins + bin[j], 1u) : 0;
    }
    __syncthreads();
    constexpr int kOwn = kBins / kThreads;
    uint32_t c[kOwn], s = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) s += c[i] = bins[tid * kOwn + i];
    uint32_t run = block_scan(s, sh.count_parts) - s;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      bins[tid * kOwn + i] = run;
      run += c[i];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (has(j)) placed[bins[bin[j]] + at[j]] = key_of(j);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      if (!has(j)) continue;
      const int a = (int)bins[bin[j]], b = bin[j] + 1 < kBins ? (int)bins[bin[j] + 1] : n;
      rank[j] = a;
      const K mine = key_of(j);
      for (int i = a; i < b; ++i) rank[j] += placed[i] > mine;
    }
    __syncthreads();
  }
};

// A bracket's tokens in the first CTA, in their order: their weights in `list` and themselves in
// `sorted` (kRegionBytes each).  `from` and `span`: the bracket's distances.
__device__ __forceinline__ void sort_bracket(const RowState& st, Shared& sh, uint64_t* list, uint64_t* sorted, int n,
                                             float from, float span) {
  constexpr int kMine = Candidates::kMine;
  const Candidates c(list, n);
  int rank[kMine];
  const float per = (float)kBins / span;
  c.ranks(sh, list, reinterpret_cast<uint32_t*>(sorted),
          [&](int j) { return min(max((int)((st.distance(c.logit(j)) - from) * per), 0), kBins - 1); },
          [&](int j) { return c.e[j]; }, rank);
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (!c.has(j)) continue;
    list[rank[j]] = st.weight(c.logit(j)).fixed();
    sorted[rank[j]] = c.e[j];
  }
  __syncthreads();
}

// The last of them that stays: number `wanted`, or (0) the one at which the running mass, with
// `before` in front, reaches the goal.  Both masses may be off by `off` together: if that leaves
// the token open, `unsure` says so.  Written to every CTA.
__device__ __forceinline__ void cut_bracket(Shared& sh, const uint64_t* list, const uint64_t* sorted, int n,
                                            int32_t wanted, Fixed before, Fixed goal, Fixed off, uint32_t ctas) {
  constexpr int kMine = Candidates::kMine;
  const int tid = (int)threadIdx.x;
  int last = min(max(wanted, 1), n) - 1;
  bool open = n == 0;
  if (wanted == 0 && n > 0) {
    Fixed w[kMine], s = 0;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      w[j] = tid * kMine + j < n ? list[tid * kMine + j] : 0;
      s += w[j];
    }
    if (tid == 0) sh.found_lo = sh.found_hi = INT32_MAX;
    Fixed run = before + block_scan(s, sh.parts) - s;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      run += w[j];
      if (tid * kMine + j < n && run + off >= goal) atomicMin(&sh.found_lo, tid * kMine + j);
      if (tid * kMine + j < n && run >= goal + off) atomicMin(&sh.found_hi, tid * kMine + j);
    }
    __syncthreads();
    last = sh.found_hi;
    // (nothing in front of the bracket may reach the goal either)
    open = last == INT32_MAX || last != sh.found_lo || before + off >= goal;
  }
  if (tid < (int)ctas) {
    *cluster_at(&sh.unsure, (uint32_t)tid) = open ? 1 : 0;
    if (!open) {
      *cluster_at(&sh.last, (uint32_t)tid) = last;
      const uint64_t c = sorted[last];
      *cluster_at(&sh.cut, (uint32_t)tid) = Cut{key_value((uint32_t)(c >> 32)), (int32_t)~(uint32_t)c};
    }
  }
}

// The candidates' way, in the cluster's first CTA alone: n of them in `list` (sorted by nothing),
// among which are all that stay.  `whole` is the row's sum if top-p is of the whole row, off by
// 2^-21 of itself at most.  `scratch`: another kRegionBytes.
template <typename T>
__device__ __forceinline__ void short_list(const SampleParams& p, const RowState& st, Shared& sh, uint64_t* list,
                                           void* scratch, int n, float threshold, int32_t k, float top_p,
                                           bool by_count, bool by_mass, Fixed whole, int row) {
  constexpr int kMine = Candidates::kMine;
  const int tid = (int)threadIdx.x;
  const Candidates c(list, n);
  uint32_t* bins = static_cast<uint32_t*>(scratch);
  Weight w[kMine];
  bool stays[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    w[j] = c.has(j) ? st.weight(c.logit(j)) : Weight{0.0f, 0.0f};
    stays[j] = w[j].hi > 0.0f;
  }
  int rank[kMine];
  Fixed* sorted = reinterpret_cast<Fixed*>(list);
  if (by_count || by_mass) {
    const float far = fminf(st.distance(threshold), kMostLog2);
    const float per = far > 0.0f ? (float)(kBins - 1) / far : 0.0f;
    c.ranks(sh, list, bins, [&](int j) { return min(max((int)(fminf(st.distance(c.logit(j)), kMostLog2) * per), 0), kBins - 1); },
            [&](int j) { return c.e[j]; }, rank);
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (by_count) stays[j] = stays[j] && rank[j] < k;
    if (by_mass) {
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        if (c.has(j)) sorted[rank[j]] = stays[j] ? w[j].fixed<kListBits>() : 0;
      __syncthreads();
      Fixed each_w[kMine], s = 0;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        each_w[j] = tid * kMine + j < n ? sorted[tid * kMine + j] : 0;
        s += each_w[j];
      }
      const Fixed before = block_scan(s, sh.parts) - s;
      // the first rank at which the running sum reaches the goal
      auto cut_at = [&](Fixed goal) {
        __syncthreads();
        if (tid == 0) sh.found = n - 1;
        __syncthreads();
        Fixed run = before;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          run += each_w[j];
          if (tid * kMine + j < n && run >= goal) atomicMin(&sh.found, tid * kMine + j);
        }
        __syncthreads();
        return sh.found;
      };
      int last;
      if (by_count) {
        last = cut_at(top_of(block_sum(s, sh), top_p));
      } else {
        constexpr int kFiner = kListBits - kFixedBits;  // (the goal is at most the list's sum)
        const Fixed off = (whole >> 21) + (1 << 14);
        last = cut_at(top_of(whole - off, top_p) << kFiner);
        if (last != cut_at(top_of(whole + off, top_p) << kFiner)) {
          // the row's sum from whole weights, by this CTA alone
          const T* z = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
          Sum all;
#pragma unroll 4
          for (int32_t v = tid; v < p.vocab; v += kThreads) all.add(st.weight(clean(to_f32(z[v]))));
          last = cut_at(top_of(block_sum(all.value(), sh), top_p) << kFiner);
        }
      }
#pragma unroll
      for (int j = 0; j < kMine; ++j) stays[j] = stays[j] && rank[j] <= last;
      __syncthreads();
    }
  }
  if (sh.rules.min_p > 0.0f) {
    const float least = fminf(sh.rules.min_p, 1.0f);
#pragma unroll
    for (int j = 0; j < kMine; ++j) stays[j] = stays[j] && (w[j].hi > least || (w[j].hi == least && w[j].lo >= 0.0f));
  }
  // in the order of the index: the largest ~token comes first
  const int down = max(0, 32 - __clz(p.vocab - 1) - 11);  // 2^11 bins
  c.ranks(sh, list, bins, [&](int j) { return c.token(j) >> down; }, [&](int j) { return (uint32_t)c.e[j]; }, rank);
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (c.has(j)) sorted[rank[j]] = stays[j] ? w[j].fixed<kListBits>() : 0;
  __syncthreads();
  Fixed each_w[kMine], s = 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    each_w[j] = tid * kMine + j < n ? sorted[tid * kMine + j] : 0;
    s += each_w[j];
  }
  if (tid == 0) sh.found = INT32_MAX, sh.found_lo = -1;
  const Fixed kept = block_sum(s, sh);
  const float u = p.random[row];
  const Fixed goal = drawn_of(kept, u);
  Fixed run = block_scan(s, sh.parts) - s;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    run += each_w[j];
    if (each_w[j] > 0) {
      if (run > goal) atomicMin(&sh.found, tid * kMine + j);
      atomicMax(&sh.found_lo, tid * kMine + j);
    }
  }
  // at the ends of u's range the first and the last that stay, however small their weights
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (stays[j] && !(u > 0.0f)) atomicMin(&sh.found, rank[j]);
    if (stays[j] && u >= 1.0f) atomicMax(&sh.found_lo, rank[j]);
  }
  __syncthreads();
  const int at = sh.found != INT32_MAX ? sh.found : sh.found_lo;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (c.has(j) && rank[j] == at) {
      p.tokens[row] = c.token(j);
      if (p.probs) p.probs[row] = quotient(w[j], kept >> (kListBits - kFixedBits));
    }
}

// The draw by short weights: where the running sum passes u times the whole.  `mine`: this CTA's
// sum, and sh.parts its warps'; listing: some tokens do not stay.  False: the sums are too near to
// say.
template <typename T>
__device__ __forceinline__ bool rough_draw(const SampleParams& p, const Part<T>& part, const RowState& st, Shared& sh,
                                           int turn, bool listing, Fixed mine) {
  constexpr int V = Part<T>::V;
  const int tid = (int)threadIdx.x, row = part.row;
  const uint32_t ctas = (uint32_t)p.cluster, rank = cluster_ctarank();
  const float u = p.random[row];
  if (tid < (int)ctas) *cluster_at(&sh.slots[turn][rank], (uint32_t)tid) = mine;
  cluster_barrier();
  Fixed whole = 0;
  for (uint32_t c = 0; c < ctas; ++c) whole += sh.slots[turn][c];
  const Fixed goal = drawn_of(whole, u);
  Fixed before = 0, run = 0;
  int owner = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const Fixed of = sh.slots[turn][c];
    if (of > 0 && run <= goal) owner = (int)c, before = run;
    run += of;
  }
  if (owner == (int)rank) {
    int w_at = 0;
    run = before;
    for (int w = 0; w < kWarps; ++w) {
      const Fixed of = sh.parts[w];
      if (of > 0 && run <= goal) w_at = w, before = run;
      run += of;
    }
    const Fixed of_warp = sh.parts[w_at];
    const int32_t a = part.first_of(w_at), b = part.first_of(w_at + 1);
    const int32_t each_q = (b - a + kThreads - 1) / kThreads;
    const int32_t qa = a + tid * each_q, qb = min(qa + each_q, b);
    auto weight_of = [&](float z, int32_t v) {
      bool near = false;
      return Weight{!listing || st.inside(clean(z), v) ? st.rough_kept(z, near) : 0.0f, 0.0f};
    };
    Fixed sum = 0;
    for (int32_t q = qa; q < qb; ++q) {
      float z[V];
      part.vector(q, z);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += weight_of(z[j], part.token(q) + j).fixed();
    }
    if (tid == 0) sh.found = -1;
    run = before + block_scan(sum, sh.parts) - sum;  // (has the barriers)
    if (sum > 0 && run <= goal) atomicMax(&sh.found, tid);
    __syncthreads();
    if (sh.found < 0 && tid == 0)  // (weights that vanish one by one)
      for (uint32_t c = 0; c < ctas; ++c) *cluster_at(&sh.near_draw, c) = 1;
    if (tid == sh.found) {
      int32_t token = -1;
      float logit = 0.0f;
      Fixed from = 0, upto = 0;
      for (int32_t q = qa; q < qb; ++q) {
        float z[V];
        part.vector(q, z);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const Fixed of = weight_of(z[j], part.token(q) + j).fixed();
          if (of > 0 && run <= goal) token = part.token(q) + j, logit = z[j], from = run, upto = run + of;
          run += of;
        }
      }
      // Is the goal in this token's part for certain?  Each weight is off by d, 2^-21 of itself at
      // most, with its part of the sums' roundings, and by the same in the running sum up to here
      // (u of the whole) and in the whole: their errors are (1 - u) d of what is in front and u d
      // of the rest, 2 (1 - u) 2^-21 of the goal together.  Within the warp the weights are added
      // up once more, another way; and there are the lanes' roundings.
      const float rest = 1.0f - u + 0x1p-20f;
      const Fixed off = ((rest < 1.0f ? share_of(goal, rest, true) : goal) >> 20) + (of_warp >> 21) + (1 << 15);
      const bool sure = from + off <= goal && goal + off < upto;
      if (sure) {
        p.tokens[row] = token;
        if (p.probs) p.probs[row] = quotient(st.weight(clean(logit)), whole);
      } else {
        for (uint32_t c = 0; c < ctas; ++c) *cluster_at(&sh.near_draw, c) = 1;
      }
    }
  }
  cluster_barrier();
  return sh.near_draw == 0;
}

// Limits that the list does not hold: the logits counted by their distance from the largest, which
// brackets the last token that stays; what lies in the bracket is sorted.  The masses are
// estimates, of a bin its middle's weight and the sum of its logits' places, good to some 10^-5 of
// the whole (without the places, off by a spread's share of the root of the squares, brackets
// were too long where p is near 1 and too short among equal logits: 64 rows of 128256 with p 0.99
// 219 us, bf16 with 0.9 130); the decision is made by the short weights' sum before the bracket.
// Every CTA of the cluster comes here, or none.
template <typename T>
__device__ __noinline__ void wide_row(const SampleParams& p, const Part<T>& given, RowState st, Shared& sh,
                                      uint32_t* region, uint64_t* list, int turn, Fixed row_sum) {
  constexpr int V = Part<T>::V;
  const Part<T> part = given;  // (in registers)
  const int tid = (int)threadIdx.x, lane = tid & 31;
  const uint32_t ctas = (uint32_t)p.cluster, rank = cluster_ctarank();
  const int32_t k = sh.rules.top_k;
  const float top_p = sh.rules.top_p, min_p = sh.rules.min_p;
  const bool by_count = k >= 1 && k < p.vocab, by_mass = top_p < 1.0f;
  uint64_t* own = reinterpret_cast<uint64_t*>(region);
  if (by_count && by_mass) {
    exact_row<T>(p, given, st, sh, region, turn);
    return;
  }
  bool summed = false;  // sh.warp_sums holds the warps' sums of what stays
  if (by_count || by_mass) {
    uint32_t* counts = region;
    int32_t* places = reinterpret_cast<int32_t*>(region + kWideBins);  // sums of 4096 times a logit's place in its bin
    uint32_t* sums = reinterpret_cast<uint32_t*>(list);                // of all CTAs, in the first one
    float* place_sums = reinterpret_cast<float*>(sums + kWideBins);
    const Fixed goal = by_mass ? top_of(row_sum, top_p) : 0;
    const float whole_f = to_float(row_sum), goal_f = to_float(goal);
    // (behind this distance lies less than half of what top-p leaves out)
    const float reach = by_count ? kMostLog2
                                 : fminf(fmaxf(__log2f((float)p.vocab) + 1.0f - __log2f(fmaxf(whole_f - goal_f, 1e-6f)), 1.0f), kMostLog2);
    const float per = (float)kWideBins / reach;
    auto bin_of = [&](float z) {  // kWideBins: behind all of them
      const float t = st.distance(z) * per;
      return t < (float)kWideBins ? max((int)t, 0) : kWideBins;  // (NaN: behind)
    };
    for (int i = tid; i < kWideBins; i += kThreads) counts[i] = 0, places[i] = 0;
    if (tid == 0) sh.mine = 0, sh.listed = 0;
    __syncthreads();
    part.each([&](float z, int32_t) {
      const int b = bin_of(z);
      if (b >= kWideBins) return;
      atomicAdd(counts + b, 1u);
      if (by_mass) atomicAdd(places + b, __float2int_rn((st.distance(z) * per - ((float)b + 0.5f)) * 4096.0f));
    });
    cluster_barrier();
    {
      // a share of the bins for each CTA, in the first one's memory
      const int share = kWideBins / (int)ctas;
      for (int i = tid; i < share; i += kThreads) {
        const int b = (int)rank * share + i;
        uint32_t c = 0;
        float f = 0.0f;
        for (uint32_t o = 0; o < ctas; ++o) {
          c += *cluster_at(counts + b, o);
          f += (float)*cluster_at(places + b, o);
        }
        *cluster_at(sums + b, 0u) = c;
        *cluster_at(place_sums + b, 0u) = f;
      }
    }
    cluster_barrier();
    if (rank == 0) {
      constexpr int kMine = kWideBins / kThreads;
      uint32_t c[kMine], cs = 0;
      float m[kMine], mass = 0.0f;
      const float ln2_per = 0.69314718f / per;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int b = tid * kMine + i;
        c[i] = sums[b];
        cs += c[i];
        // 2^(-f / per) for places f around the bin's middle, to the second order of evenly spread ones
        m[i] = exp2f(-((float)b + 0.5f) / per) *
               ((float)c[i] * (1.0f + ln2_per * ln2_per / 24.0f) - place_sums[b] * (ln2_per / 4096.0f));
        mass += m[i];
      }
      if (tid == 0) sh.found_lo = sh.found_hi = kWideBins - 1;
      uint32_t run_c = block_scan(cs, sh.count_parts) - cs;
      float run = block_scan(mass, sh.low_parts) - mass;
      const float margin = 3e-5f * whole_f;
      const uint32_t first_c = run_c;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int b = tid * kMine + i;
        run_c += c[i];
        run += m[i];
        if (by_count ? run_c >= (uint32_t)k : run + margin >= goal_f) atomicMin(&sh.found_lo, b);
        if (by_count ? run_c >= (uint32_t)k : run - margin >= goal_f) atomicMin(&sh.found_hi, b);
      }
      __syncthreads();
      run_c = first_c;
      const int lo = sh.found_lo, hi = sh.found_hi;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int b = tid * kMine + i;
        if (b == lo) sh.ends[0] = run_c;
        run_c += c[i];
        if (b == hi) sh.ends[1] = run_c;
      }
      if (tid == kThreads - 1) sh.base = run_c;
      __syncthreads();
      if (tid == 0) {
        const Bracket br{lo, hi, 0, 0, 0.0f, 0.0f, sh.ends[0], sh.ends[1] - sh.ends[0], sh.base};
        for (uint32_t o = 0; o < ctas; ++o) *cluster_at(&sh.bracket, o) = br;
      }
    }
    cluster_barrier();
    const Bracket br = sh.bracket;
    if (br.count > kList) {
      exact_row<T>(p, given, st, sh, region, turn);
      return;
    }
    if (!by_count || br.all > (uint32_t)k) {
      Sum ahead;
      part.each([&](float z, int32_t v) {
        const int b = bin_of(z);
        if (b > br.hi || b >= kWideBins) return;
        if (b >= br.lo) {
          const uint32_t at = atomicAdd(&sh.mine, 1u);
          if (at < kList) own[at] = (uint64_t)order_key(z) << 32 | (uint32_t)~v;
        } else {
          ahead.add({st.rough(z), 0.0f});
        }
      });
      const Fixed mine_ahead = block_sum(ahead.value(), sh);
      if (tid < kWarps) sh.warp_sums[tid] = sh.parts[tid];
      const uint32_t count = min(sh.mine, (uint32_t)kList);
      if (tid == 0) sh.base = atomicAdd(cluster_at(&sh.listed, 0u), count);
      if (tid < (int)ctas) *cluster_at(&sh.slots[turn][rank], (uint32_t)tid) = mine_ahead;
      __syncthreads();
      uint64_t* to = cluster_at(list, 0u);
      for (uint32_t i = (uint32_t)tid; i < count; i += kThreads)
        if (sh.base + i < kList) to[sh.base + i] = own[i];
      cluster_barrier();
      Fixed before = 0;
      for (uint32_t o = 0; o < ctas; ++o) before += sh.slots[turn][o];
      turn ^= 1;
      uint64_t* sorted = reinterpret_cast<uint64_t*>(region);
      const int n = (int)br.count;
      if (rank == 0) {
        sort_bracket(st, sh, list, sorted, n, (float)br.lo / per, (float)(br.hi - br.lo + 1) / per);
        // The row's sum is off by 2^-22 + 2^-24 of each weight, and 3 2^-24 of it for the sums of
        // eight; the one in front, which is part of it, by the former, the same of each weight.
        const float share = fminf(top_p, 1.0f), front = to_float(before), all = to_float(row_sum);
        const float off = 1.01f * 0x1p-22f * (1.25f * ((1.0f - share) * front + share * fmaxf(all - front, 0.0f)) + 0.75f * share * all);
        cut_bracket(sh, list, sorted, n, by_count ? k - (int32_t)br.before : 0, before, goal,
                    (Fixed)__float2ll_ru(off * (float)(1ull << kFixedBits)) + (1 << 14), ctas);
      }
      cluster_barrier();
      const Pairs pairs(st);
      if (sh.unsure && by_mass && n > 0 && pairs.usable) {
        // the same from whole weights: the row's sum and the mass before the bracket
        Sum2 every, first;
        for (int32_t q = part.q0 + lane; q < part.q1; q += 32) {
          float z[V];
          part.vector(q, z);
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const Weights2 w = pairs.weights(z[j], z[j + 1], true, true);
            every.add(w);
            const bool a = bin_of(z[j]) < br.lo, b = bin_of(z[j + 1]) < br.lo;
            if (__any_sync(__activemask(), a || b)) {
              float h0, h1, l0, l1;
              parts_of(w.hi, h0, h1);
              parts_of(w.lo, l0, l1);
              first.add({two(a ? h0 : 0.0f, b ? h1 : 0.0f), two(a ? l0 : 0.0f, b ? l1 : 0.0f)});
            }
          }
        }
        const Fixed mine_first = block_sum(first.value(), sh);
        const Fixed mine_every = block_sum(every.value(), sh);
        if (tid < (int)ctas) {
          *cluster_at(&sh.slots[turn][rank], (uint32_t)tid) = mine_every;
          *cluster_at(&sh.more_slots[rank], (uint32_t)tid) = mine_first;
        }
        cluster_barrier();
        Fixed sum = 0;
        before = 0;
        for (uint32_t o = 0; o < ctas; ++o) sum += sh.slots[turn][o], before += sh.more_slots[o];
        turn ^= 1;
        if (rank == 0) cut_bracket(sh, list, sorted, n, 0, before, top_of(sum, top_p), 0, ctas);
        cluster_barrier();
      }
      if (sh.unsure) {
        exact_row<T>(p, given, st, sh, region, turn);
        return;
      }
      st.cut_z = sh.cut.z;
      st.cut_v = sh.cut.v;
      if (!(min_p > 0.0f)) {
        // what stays: the sums before the bracket, and of the bracket the first ones
        const Fixed* weights = cluster_at(list, 0u);
        const uint64_t* tokens = cluster_at(sorted, 0u);
        for (int i = tid; i <= sh.last; i += kThreads) {
          const int32_t at = (int32_t)~(uint32_t)tokens[i] - part.v0;
          if (at < 0 || at >= part.n) continue;
          const int32_t q = (at + part.shift) / V;
          int w = (int)((int64_t)q * kWarps / part.vectors);
          while (part.first_of(w + 1) <= q) ++w;
          while (part.first_of(w) > q) --w;
          atomicAdd((unsigned long long*)&sh.warp_sums[w], (unsigned long long)weights[i]);
        }
        summed = true;
      }
    }
  }
  Fixed mine = 0;
  if (summed) {
    __syncthreads();
    if (tid < kWarps) sh.parts[tid] = sh.warp_sums[tid];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mine += sh.warp_sums[w];
  } else {
    if (min_p > 0.0f) st.min_p = fminf(min_p, 1.0f);
    // the short weights of what stays
    Sum all;
    bool near = false;
    part.each([&](float z, int32_t v) {
      if (st.inside(z, v)) all.add({st.rough_kept(z, near), 0.0f});
    });
    if (near)
      for (uint32_t o = 0; o < ctas; ++o) *cluster_at(&sh.near_draw, o) = 1;
    mine = block_sum(all.value(), sh);
  }
  if (!rough_draw<T>(p, part, st, sh, turn, true, mine)) exact_draw<T>(p, given, st, sh, turn ^ 1);
}

// 2^(-j / 64), hi and lo.
struct Powers {
  float v[2 * kTable];
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p,
                                                             const __grid_constant__ Powers powers) {
  constexpr int V = Part<T>::V;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  float* table = reinterpret_cast<float*>(smem);
  uint32_t* region = reinterpret_cast<uint32_t*>(smem + kTableBytes);
  uint64_t* list = reinterpret_cast<uint64_t*>(smem + kTableBytes + kRegionBytes);
  const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ctas = (uint32_t)p.cluster, rank = cluster_ctarank();
  int row = (int)(blockIdx.x / ctas), next = row + p.ahead;

  // (every CTA of the cluster has to have started before another writes to its memory)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  for (int i = tid; i < 2 * kTable * kCopies; i += kThreads) table[i] = powers.v[i / kCopies];
  if (tid == 0) sh.listed = sh.mine = 0, sh.unsure = sh.near_draw = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  if (p.ordered) {
    const int2 rows = in_order(p, row, next, sh);
    row = rows.x;
    next = rows.y;
  }

  int32_t k = p.top_k ? p.top_k[row] : 0;
  float top_p = p.top_p ? p.top_p[row] : 1.0f;
  bool by_count = k >= 1 && k < p.vocab, by_mass = top_p < 1.0f;
  if (tid == 0) {
    const float temperature = p.temperature ? p.temperature[row] : 1.0f;
    // log2(e) / T: the quotient, and what its product with T lacks
    constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.92596299112661746887e-8f;
    const float q = __fdiv_rn(kLog2eHi, temperature);
    const float lack = __fdiv_rn(fmaf(-q, temperature, kLog2eHi) + kLog2eLo, temperature);
    sh.own_rules = {q, isfinite(q) && isfinite(lack) ? lack : 0.0f, !(temperature > 0.0f), k, top_p,
                    p.min_p ? p.min_p[row] : 0.0f};
  }

  Part<T> part;
  part.row = row;
  part.v0 = min((int32_t)rank * p.slice, p.vocab);
  part.n = min(p.slice, p.vocab - part.v0);
  part.in = static_cast<const T*>(p.logits) + (int64_t)row * p.stride + part.v0;
  part.slice = reinterpret_cast<T*>(smem + kFixedSmem);
  part.shift = part.n > 0 ? (int32_t)((reinterpret_cast<uintptr_t>(part.in) / sizeof(T)) % V) : 0;
  part.vectors = (part.n + part.shift + V - 1) / V;
  part.q0 = part.first_of(warp), part.q1 = part.first_of(warp + 1);
  part.resident = p.resident != 0;

  // The row that will run here after this one is brought into L2 meanwhile, so that memory is read
  // also while the rows here are worked on.  8 KB by each instruction, so that several threads ask for a
  // slice: nothing requires that size, and larger pieces have not been measured.
  if (next < p.rows && part.n > 0) {
    constexpr uintptr_t kAhead = 8192;
    const uintptr_t from = reinterpret_cast<uintptr_t>(part.in + (int64_t)(next - row) * p.stride);
    const uintptr_t a = (from + 15) & ~(uintptr_t)15, b = (from + (uintptr_t)part.n * sizeof(T)) & ~(uintptr_t)15;
    for (uintptr_t at = a + (uintptr_t)tid * kAhead; at < b; at += kThreads * kAhead)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"((uint32_t)min(kAhead, b - at)) : "memory");
  }

  // ---------------------------------------------------------------- the largest --
  float best = -__builtin_huge_valf();
  {
    constexpr int kRun = 4;
    for (int32_t q = part.q0 + lane; q < part.q1; q += 32 * kRun) {
      Pack<T, V> x[kRun];
#pragma unroll
      for (int r = 0; r < kRun; ++r)
        if (q + 32 * r < part.q1) x[r] = part.from_memory(q + 32 * r);
#pragma unroll
      for (int r = 0; r < kRun; ++r) {
        if (q + 32 * r >= part.q1) break;
        if (part.resident) *reinterpret_cast<Pack<T, V>*>(part.slice + (q + 32 * r) * V) = x[r];
        best = fmaxf(best, largest(x[r]));
      }
    }
  }
  // the candidates' threshold: the wanted number of them, and what share of the lanes (of 32 that
  // many) has one
  const bool few_tokens = p.vocab <= kList;
  if ((by_count || by_mass) && !few_tokens) {
    const float wanted = by_count ? fminf(1.3f * (float)k + 60.0f, 1750.0f) : 1400.0f;
    const float share = 1.0f - __expf(-wanted / (float)(kThreads * ctas));
    const int q = min(max((int)ceilf(0.33f + 32.0f * share), 1), 31);
    float x = best;  // sorted over the warp, the largest first
#pragma unroll
    for (int len = 2; len <= 32; len *= 2)
#pragma unroll
      for (int gap = len / 2; gap > 0; gap /= 2) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, x, gap);
        x = ((lane & gap) == 0) == ((lane & len) == 0) ? fmaxf(x, o) : fminf(x, o);
      }
    x = __shfl_sync(0xFFFFFFFFu, x, q - 1);
    if (lane == 0) sh.warp_quantile[warp] = x;
  }
  for (int off = 16; off > 0; off >>= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, off));
  if (lane == 0) sh.warp_best[warp] = best;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
#pragma unroll
  for (int w = 0; w < kWarps; ++w) best = fmaxf(best, sh.warp_best[w]);
  if (warp == 0 && (by_count || by_mass) && !few_tokens) {
    // the middle one of the warps'
    int above = 0;
    const float x = sh.warp_quantile[lane % kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float o = sh.warp_quantile[w];
      above += o > x || (o == x && w < lane);
    }
    if (lane < kWarps && above == kWarps / 2)
      for (uint32_t c = 0; c < ctas; ++c) *cluster_at(&sh.quantile[rank], c) = x;
  }
  if (tid < (int)ctas) {
    *cluster_at(&sh.best[rank], (uint32_t)tid) = best;
    if (rank == 0) *cluster_at(&sh.rules, (uint32_t)tid) = sh.own_rules;
  }
  cluster_barrier();
  k = sh.rules.top_k;
  top_p = sh.rules.top_p;
  const float min_p = sh.rules.min_p;
  by_count = k >= 1 && k < p.vocab, by_mass = top_p < 1.0f;
  for (uint32_t c = 0; c < ctas; ++c) best = fmaxf(best, sh.best[c]);
  best += 0.0f;  // (not -0)
  const bool writer = rank == 0 && tid == 0;
  if (best == -__builtin_huge_valf()) {
    if (writer) {
      p.tokens[row] = -1;
      if (p.probs) p.probs[row] = 0.0f;
    }
    return;
  }
  if (sh.rules.greedy) {
    if (tid == 0) sh.found = INT32_MAX;
    __syncthreads();
    part.each([&](float z, int32_t v) {
      if (z == best) atomicMin(&sh.found, v);
    });
    __syncthreads();
    if (tid == 0) *cluster_at(&sh.first[rank], 0u) = sh.found;
    cluster_barrier();
    if (writer) {
      int32_t first = sh.first[0];
      for (uint32_t c = 1; c < ctas; ++c) first = min(first, sh.first[c]);
      p.tokens[row] = first;
      if (p.probs) p.probs[row] = 1.0f;
    }
    return;
  }

  RowState st;
  st.m = best;
  st.scale_hi = sh.rules.scale_hi;
  st.scale_lo = sh.rules.scale_lo;
  st.cut_z = -__builtin_huge_valf();
  st.cut_v = INT32_MAX;
  st.min_p = 0.0f;
  st.table = table + (lane & (kCopies - 1));
  if (!isfinite(best) || !isfinite(st.scale_hi)) {
    exact_row<T>(p, part, st, sh, region, 0);
    return;
  }

  // ------------------------------------------------------------- one pass over the row --
  // LIST: candidates; TOTAL: the short weights' sum, and the candidates'.
  const bool listing = by_count || by_mass || min_p > 0.0f;
  float threshold = -__builtin_huge_valf();
  if (few_tokens) {
  } else if (by_count || by_mass) {
    threshold = middle(sh.quantile, (int)ctas);
  } else if (min_p > 0.0f) {
    // weights of min_p and more, and a little below
    threshold = best - (1.0001f * fmaxf(-__log2f(fminf(min_p, 1.0f)), 0.0f) + 0.001f) / st.scale_hi;
  }
  uint64_t* own = reinterpret_cast<uint64_t*>(region);
  auto pass = [&](auto with_list, auto with_total, Sum& all, Sum& chosen) {
    part.vectors_of([&](const float (&z)[V], int32_t q) {
      if constexpr (decltype(with_list)::value) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (z[j] >= threshold && z[j] > -__builtin_huge_valf()) {
            const uint32_t at = atomicAdd(&sh.mine, 1u);
            if (at < kList) own[at] = (uint64_t)order_key(z[j] + 0.0f) << 32 | (uint32_t)~(part.token(q) + j);
            if constexpr (decltype(with_total)::value) chosen.add({st.rough(z[j]), 0.0f});
          }
        }
      }
      if constexpr (decltype(with_total)::value) {
        float w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = st.rough(z[j]);
#pragma unroll
        for (int gap = V / 2; gap > 0; gap /= 2)
#pragma unroll
          for (int j = 0; j < gap; ++j) w[j] += w[j + gap];
        all.add({w[0], 0.0f});
      }
    });
  };
  Sum all, chosen;
  using Yes = std::true_type;
  using No = std::false_type;
  if (!listing) pass(No{}, Yes{}, all, chosen);
  else if (by_mass && !by_count) pass(Yes{}, Yes{}, all, chosen);
  else pass(Yes{}, No{}, all, chosen);
  int turn = 0;

  if (listing) {
    const Fixed mine_chosen = block_sum(chosen.value(), sh);
    const Fixed mine_all = block_sum(all.value(), sh);
    const uint32_t count = sh.mine;
    if (tid == 0) sh.base = atomicAdd(cluster_at(&sh.listed, 0u), count);
    if (tid < (int)ctas) {
      *cluster_at(&sh.counts[rank], (uint32_t)tid) = count;
      *cluster_at(&sh.slots[turn][rank], (uint32_t)tid) = mine_all;
      *cluster_at(&sh.more_slots[rank], (uint32_t)tid) = mine_chosen;
    }
    __syncthreads();
    uint64_t* to = cluster_at(list, 0u);
    for (uint32_t i = (uint32_t)tid; i < min(count, (uint32_t)kList); i += kThreads)
      if (sh.base + i < kList) to[sh.base + i] = own[i];
    cluster_barrier();
    uint32_t n = 0;
    Fixed whole = 0, listed = 0;
    for (uint32_t c = 0; c < ctas; ++c) n += sh.counts[c], whole += sh.slots[turn][c], listed += sh.more_slots[c];
    turn ^= 1;
    bool enough = n <= kList;
    if (threshold > -__builtin_huge_valf()) {
      if (by_count) enough = enough && n >= (uint32_t)k;
      // (both sums are within 2^-21 of themselves)
      else if (by_mass) enough = enough && listed - (listed >> 20) >= top_of(whole + (whole >> 20), top_p);
    }
    if (enough) {
      if (rank == 0)
        short_list<T>(p, st, sh, list, region, (int)n, threshold, k, top_p, by_count, by_mass, whole, row);
    } else {
      wide_row<T>(p, part, st, sh, region, list, turn, whole);
    }
    return;
  }
  if (!rough_draw<T>(p, part, st, sh, 0, false, block_sum(all.value(), sh))) exact_draw<T>(p, part, st, sh, 1);
}

template <typename T>
cudaError_t launch(SampleParams& p, int sms, cudaStream_t stream) {
  // Clusters as large as let all rows run at once, of slices of at least 2048 logits; more rows than
  // that in clusters of up to four, of slices of at least 16384 (256 x 128256 fp32 with mixed limits
  // 136 us in clusters of four when of two it took 184, alone 298).  (Two CTAs on an SM; clusters of 4
  // and 8 leave some SMs of each processing cluster without: 37 rows of 50257 in clusters of 8, one
  // of which waits, 26 us, in clusters of 4 17; 72 rows of 128256 fp32, greedy, in clusters of 4 15.4
  // us, 76 25.6.)
  constexpr int kPerSm = 2;
  auto at_once = [&](int c) { return c == 8 ? sms * 32 / 152 : c == 4 ? sms * 72 / 152 : kPerSm * sms / c; };
  p.cluster = 1;
  while (p.cluster < kMaxCluster && p.rows <= at_once(2 * p.cluster) && p.vocab > p.cluster * 2048) p.cluster *= 2;
  while (p.cluster < 4 && p.vocab > p.cluster * 16384) p.cluster *= 2;
  p.ahead = at_once(p.cluster);
  p.ordered = p.top_p != nullptr && p.rows > p.ahead && p.rows <= kMostOrdered;
  constexpr int V = 16 / (int)sizeof(T);
  p.slice = (int32_t)(((int64_t)p.vocab + p.cluster - 1) / p.cluster);
  const size_t bytes = ((size_t)p.slice + 2 * V) * sizeof(T) / 16 * 16;
  // A slice stays in shared memory where two CTAs of such an SM leave L1 something, or where there is
  // one, else it is read from L2 (256 x 128256 bf16, clusters of 4, slices of 64 KB, greedy 60 us from
  // L2, 68 with them kept; 64 x 50257 fp32, 50 KB, 8.2 and 7.7; 8 rows of 128256 fp32 in clusters of 8,
  // 64 KB, one CTA on an SM, 7.0 and 6.2).
  constexpr size_t kMost = 111 * 1024;
  const bool alone = (int64_t)p.rows * p.cluster <= sms;
  p.resident = bytes <= (alone ? kMost - kFixedSmem : 56 * 1024);
  const size_t smem = kFixedSmem + (p.resident ? bytes : 0);
  auto kernel = sample_kernel<T>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.rows * p.cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static const Powers powers = [] {
    Powers w;
    for (int j = 0; j < kTable; ++j) {
      const double e = std::exp2(-(double)j / kTable);
      w.v[2 * j] = (float)e;
      w.v[2 * j + 1] = (float)(e - (double)(float)e);
    }
    return w;
  }();
  return cudaLaunchKernelEx(&cfg, kernel, p, powers);
}

}  // namespace

cudaError_t launch_sample(SampleParams p, int elem, int sms, cudaStream_t stream) {
  switch (elem) {
    case kElemF16: return launch<__half>(p, sms, stream);
    case kElemBF16: return launch<__nv_bfloat16>(p, sms, stream);
    case kElemF32: return launch<float>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gb300

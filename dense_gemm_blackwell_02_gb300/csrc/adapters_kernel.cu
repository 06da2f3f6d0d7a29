// Low-rank adapters beside a shared projection, a different one for every row:
//     Y[i] = W . X[i] + s * Up[a] . (Down[a] . X[i]),   a = row_adapter[i]
// for many rows.  The kernel here forms u[i] = s * Down[a] . X[i] in binary32; the GEMM then
// appends Up[a] . u[i] to every tile (ADAPT in gemm_kernel.cuh), so that Y is written once,
// rounded once, and nothing of its size is read or written besides.
//
// The rows are taken 128 at a time in their own order, whatever adapters they name.  A tile's
// distinct adapters are numbered (slots), and the tensor cores multiply the whole tile by
// each of them, every adapter into accumulator columns of its own; a row then takes the
// columns of the one it names.  So rows need no sorting, nothing of one adapter enters
// another row's sums (infinities and NaN included), and the surplus products cost nothing
// that is scarce: X, read once (134 MB at 8192 x 8192, 20 us of HBM), bounds the kernel.
//
// Measured with the product: 8192 x 10240 x 8192, 12 adapters of rank 64 (prompts of some 700
// rows, so that a tile multiplies by one or two), bf16, 760 to 825 us as the power cap has it,
// 1690 to 1830 TFLOP/s (880 to 910 us when called back to back for seconds); 2050 x 4096 x 4096,
// 6 of rank 32, fp16, 65 to 66 us, where the product alone takes 46 and rows without adapters 51.  Of the 15 us that this kernel has there, the first K block is in
// shared memory after 5.6, the MMAs are done after 9, and the clusters' sums and the stores of
// u take the rest: the latency of its steps bounds it, not X's 17 MB.  Asking for X ahead of
// the rows' adapters (into L2) delays the first K block by 2 us.
//
// u leaves as 16-bit parts, in fp16 times a power of two that brings the row into its range,
// with what is far below the row's largest in a second window (RowFactor): one part alone would round u to 8 or 11 bits, an error of the size of Y's own
// rounding (how many, and what they leave: u_parts).  u itself goes along in binary32 for the
// rows and columns that parts do not serve.
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "umma.cuh"
#include "wait.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 192;  // warp 0 copies, warp 1 multiplies, warps 2..5 take results out
constexpr int kMaxStages = 8;
constexpr uint32_t kRowBytes = 128;                          // 64 values of K
constexpr uint32_t kTileBytes = kAdapterRows * kRowBytes;    // a 128 x 64 operand tile

// A tile's rows by adapter.
struct TileSlots {
  alignas(16) int32_t id[kAdapterRows];  // the row's adapter, or -1
  int32_t adapter[kAdapterRows];         // of each slot, in the order of first rows
  int16_t slot[kAdapterRows];            // of each row, or -1
  int16_t order[kAdapterRows];           // rows with an adapter, slot after slot
  int16_t start[kAdapterRows + 1];       // of each slot in `order`
  float scale[kAdapterRows];             // of each slot's adapter
  int32_t warp_firsts[4];
  int32_t slots;
};

// All threads of the CTA call it; the first 128 do the work.
__device__ void number_slots(TileSlots& ts, const AdapterParams& p, int32_t row0) {
  const int t = (int)threadIdx.x;
  int32_t a = -1;
  if (t < kAdapterRows) {
    if (row0 + t < p.M) {
      a = p.row_adapter[row0 + t];
      if (a >= p.count) {  // not followed
        record_bad_index(p.status, kSiteRowAdapter);
        a = -1;
      }
      if (a < 0) a = -1;
    }
    ts.id[t] = a;
  }
  __syncthreads();
  int first = kAdapterRows, before = 0, total = 0;
  bool is_first = false;
  if (t < kAdapterRows) {
    if (a >= 0) {
      for (int j = 0; j < kAdapterRows; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(ts.id + j);
        const int32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (w[k] == a) {
            first = min(first, j + k);
            before += j + k < t ? 1 : 0;
            ++total;
          }
      }
      is_first = first == t;
    }
    const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, is_first);
    if ((t & 31) == 0) ts.warp_firsts[t >> 5] = __popc(firsts);
    if (is_first) ts.slot[t] = (int16_t)__popc(firsts & ((1u << (t & 31)) - 1u));
  }
  __syncthreads();
  if (t < kAdapterRows && is_first) {
    int s = ts.slot[t];
    for (int w = 0; w < (t >> 5); ++w) s += ts.warp_firsts[w];
    ts.slot[t] = (int16_t)s;
    ts.adapter[s] = a;
    ts.start[s + 1] = (int16_t)total;
  }
  if (t == 0) {
    ts.start[0] = 0;
    ts.slots = ts.warp_firsts[0] + ts.warp_firsts[1] + ts.warp_firsts[2] + ts.warp_firsts[3];
  }
  __syncthreads();
  const int slot = t < kAdapterRows && a >= 0 ? ts.slot[first] : -1;
  if (t < 32) {  // counts -> starts: four per lane, then across the warp
    int c[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = 4 * t + k;
      sum += s < ts.slots ? ts.start[s + 1] : 0;
      c[k] = sum;
    }
    int run = sum;
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, run, off);
      if (t >= off) run += o;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (4 * t + k < ts.slots) ts.start[4 * t + k + 1] = (int16_t)(run - sum + c[k]);
  }
  __syncthreads();
  if (t < kAdapterRows) {
    ts.slot[t] = (int16_t)slot;
    if (slot >= 0) ts.order[ts.start[slot] + before] = (int16_t)t;
  }
  __syncthreads();
  // (read much later, after other barriers)
  if (t < ts.slots) ts.scale[t] = p.scale ? __ldg(p.scale + ts.adapter[t]) : 1.0f;
}

// Where a CTA's barriers stand in shared memory.
struct Bars {
  uint32_t base;
  __device__ uint32_t full(uint32_t s) const { return base + 8u * s; }
  __device__ uint32_t empty(uint32_t s) const { return base + 8u * (kMaxStages + s); }
  __device__ uint32_t acc_full() const { return base + 8u * (2 * kMaxStages); }
  __device__ uint32_t acc_empty() const { return base + 8u * (2 * kMaxStages + 1); }
  __device__ uint32_t drain() const { return base + 8u * (2 * kMaxStages + 2); }
  __device__ void init() const {
    for (uint32_t s = 0; s < kMaxStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full(), 1);
    mbar_init(acc_empty(), 4);
    mbar_init(drain(), 1);
    fence_mbarrier_init();
  }
};
constexpr int kNumBars = 2 * kMaxStages + 3;

// ---------------------------------------------------------------------------- Down . X --
// A row tile belongs to a cluster of CTAs, which share its (group of adapters, K slice)
// units: as many K slices as leave every CTA one unit.  A group is what fits 128 accumulator
// columns.  The slices meet in distributed shared memory (the idle operand ring), where each
// CTA of a group adds its share of the rows, in slice order.
constexpr uint32_t kRing = 96 * 1024;  // two CTAs per SM
constexpr uint32_t kSmem = kRing + 1024;

// N values as P parts, kBlockK values apart; LOW: in the second window.
template <typename T, int N, int P, bool LOW = false>
__device__ __forceinline__ void store_parts(T* to, const float (&v)[N], const RowFactor& f) {
  struct alignas(N * sizeof(T)) { T x[N]; } part[P];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    T x[P];
    split_f32(LOW ? f.low(v[k]) : f.high(v[k]), x);
#pragma unroll
    for (int j = 0; j < P; ++j) part[j].x[k] = x[j];
  }
#pragma unroll
  for (int j = 0; j < P; ++j) *reinterpret_cast<decltype(&part[0])>(to + j * kBlockK) = part[j];
}

// The adapters of two row tiles, as the GEMM's 256-row tile takes them.
__device__ void list_tile(const AdapterParams& p, int32_t pair, TileSlots& t0, TileSlots& t1) {
  number_slots(t0, p, 2 * pair * kAdapterRows);
  number_slots(t1, p, (2 * pair + 1) * kAdapterRows);
  AdapterTile& out = p.pairs[pair];
  const int t = (int)threadIdx.x;
  const int warp = (int)warp_id(), lane = (int)lane_id();
  __shared__ int16_t place[kAdapterRows];  // of the second tile's slots in the list
  __shared__ int16_t twin[kAdapterRows];   // the second tile's slot of a first one's adapter
  if (t < kAdapterRows) {
    twin[t] = -1;
    place[t] = -1;
  }
  __syncthreads();
  for (int s = t; s < t1.slots; s += kThreads)
    for (int q = 0; q < t0.slots; ++q)
      if (t0.adapter[q] == t1.adapter[s]) place[s] = (int16_t)q, twin[q] = (int16_t)s;
  __syncthreads();
  if (t == 0) {
    int n = t0.slots;
    for (int s = 0; s < t1.slots; ++s)
      if (place[s] < 0) place[s] = (int16_t)n++;
    out.slots = n;
  }
  __syncthreads();
  if (warp < 4) {
    const int r = warp * 32 + lane, s0 = t0.slot[r], s1 = t1.slot[r];
    for (int q = 0; q < t0.slots; ++q) {
      const uint32_t m0 = __ballot_sync(0xFFFFFFFFu, s0 == q);
      const uint32_t m1 = __ballot_sync(0xFFFFFFFFu, twin[q] >= 0 && s1 == twin[q]);
      if (lane == 0) {
        out.slot[q].adapter = t0.adapter[q];
        out.slot[q].disable[warp] = ~m0;
        out.slot[q].disable[4 + warp] = ~m1;
      }
    }
    for (int q = 0; q < t1.slots; ++q) {
      if (place[q] < t0.slots) continue;
      const uint32_t m1 = __ballot_sync(0xFFFFFFFFu, s1 == q);
      if (lane == 0) {
        out.slot[place[q]].adapter = t1.adapter[q];
        out.slot[place[q]].disable[warp] = 0xFFFFFFFFu;
        out.slot[place[q]].disable[4 + warp] = ~m1;
      }
    }
  }
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// P: the parts of u.
template <typename T, int P>
__global__ void __launch_bounds__(kThreads, 2)
    adapter_down_kernel(const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmDown, const AdapterParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ TileSlots ts;
  __shared__ alignas(8) uint64_t bar_mem[kNumBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t abort_mem;
  __shared__ int32_t low_mem;  // a row that this CTA sees to has a second window
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const Bars bars{smem_addr(bar_mem)};
  const uint32_t warp = warp_id(), lane = lane_id();
  const WaitCtl ctl{p.wait_limit_ns, p.status, &abort_mem};
  const int32_t tile = (int32_t)blockIdx.x / p.ctas;
  const int32_t cta = (int32_t)blockIdx.x - tile * p.ctas;  // rank in the cluster

  if (tile >= p.tiles) {  // the clusters after the row tiles' list the adapters of pairs of them
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t pair = (int32_t)blockIdx.x - p.tiles * p.ctas;
    if (2 * pair < p.tiles)
      list_tile(p, pair, ts, *reinterpret_cast<TileSlots*>(smem_raw));
    return;
  }

  if (warp == 0 && lane == 0) {
    bars.init();
    abort_mem = 0;
    low_mem = 0;
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmDown);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_addr(&tmem_slot), kAdapterCols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  number_slots(ts, p, tile * kAdapterRows);
  const int32_t per_group = kAdapterCols / p.rank;
  const int32_t groups = (ts.slots + per_group - 1) / per_group;
  const int32_t splits = groups == 0 ? 1 : min(max(p.ctas / groups, 1), p.max_splits);
  const int32_t units = groups * splits;
  // A stage: X's rows, then the group's rows of Down; the MMA's N is a multiple of 16.
  const uint32_t n_max = ((uint32_t)(min(per_group, ts.slots) * p.rank) + 15u) & ~15u;
  const uint32_t stage_bytes = kTileBytes + n_max * kRowBytes;
  const uint32_t stages = min((uint32_t)kMaxStages, kRing / stage_bytes);
  const int32_t window = P * kBlockK * (p.rank <= kBlockK ? 1 : 2);  // of U's rows
  constexpr bool kWindows = std::is_same<T, __half>::value;
  const int32_t pitch = (kWindows ? 2 : 1) * window;
  T* U = static_cast<T*>(p.U) + (int64_t)tile * kAdapterRows * pitch;
  // value c of a row: 64 at a time, their first parts before their second ones
  auto place_of = [](int32_t c) { return (c >> 6) * P * kBlockK + (c & (kBlockK - 1)); };
  if (cta == 0 && threadIdx.x < kAdapterRows && ts.slot[threadIdx.x] < 0 &&
      tile * kAdapterRows + (int32_t)threadIdx.x < p.M) {
    p.row_scale[tile * kAdapterRows + (int32_t)threadIdx.x] = 0.0f;
    p.row_scale_low[tile * kAdapterRows + (int32_t)threadIdx.x] = 0.0f;
  }

  if (warp == 0) {
    uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    for (int32_t u = cta; ok && u < units; u += p.ctas) {
      const int32_t group = u / splits, s = u - group * splits;
      const int32_t g0 = group * per_group, n = min(per_group, ts.slots - g0);
      const int32_t kb1 = (int32_t)((int64_t)(s + 1) * p.k_blocks / splits);
      for (int32_t kb = (int32_t)((int64_t)s * p.k_blocks / splits); kb < kb1; ++kb) {
        if (!warp_wait_inl(bars.empty(stage), phase ^ 1u, ctl, kSiteAdapterEmpty)) {
          ok = false;
          break;
        }
        const uint32_t at = ring + stage * stage_bytes;
        mbar_arrive_expect_tx_elect(bars.full(stage), (uint32_t)(kAdapterRows + n * p.rank) * kRowBytes);
        tma_load_2d_elect(at, &tmX, kb * kBlockK, tile * kAdapterRows, bars.full(stage));
        for (int32_t j = 0; j < n; ++j)
          tma_load_2d_elect(at + kTileBytes + (uint32_t)(j * p.rank) * kRowBytes, &tmDown, kb * kBlockK,
                            ts.adapter[g0 + j] * p.rank, bars.full(stage));
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0)
      for (uint32_t s = 0; s < stages; ++s)
        if (armed & (1u << s)) wait_parity_drain(bars.full(s), (armed_phase >> s) & 1u, ctl);
    __syncwarp();
  } else if (warp == 1) {
    uint32_t stage = 0, phase = 0, iter = 0;
    bool ok = !p.test_stall || warp_wait(bars.drain(), 0, ctl, kSiteTestStall);
    for (int32_t u = cta; ok && u < units; u += p.ctas, ++iter) {
      const int32_t group = u / splits, s = u - group * splits;
      const int32_t n = min(per_group, ts.slots - group * per_group);
      const uint32_t idesc = p.idesc | ((((uint32_t)(n * p.rank) + 15u) >> 4) << 18);  // N >> 3 at bit 17
      if (!warp_wait_inl(bars.acc_empty(), (iter & 1u) ^ 1u, ctl, kSiteAdapterAcc)) break;
      tc_fence_after();
      const int32_t kb0 = (int32_t)((int64_t)s * p.k_blocks / splits);
      const int32_t kb1 = (int32_t)((int64_t)(s + 1) * p.k_blocks / splits);
      for (int32_t kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_inl(bars.full(stage), phase, ctl, kSiteAdapterFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = ring + stage * stage_bytes;
        umma_stage_elect<1>(tmem, smem_desc_sw128_kmajor(at), smem_desc_sw128_kmajor(at + kTileBytes),
                            idesc, kb > kb0 ? 1u : 0u, bars.empty(stage));
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      if (ok) umma_commit_elect<1>(bars.acc_full());
    }
    // every MMA has read its operands and written its columns before the ring is reused and
    // the CTA tears down
    umma_commit_elect<1>(bars.drain());
    if (lane == 0) wait_parity_drain(bars.drain(), 0, ctl);
    __syncwarp();
  } else {
    const uint32_t quarter = warp & 3u;
    const int32_t row = (int32_t)(quarter * 32 + lane);
    const int32_t slot = ts.slot[row];
    const float f = slot >= 0 && p.scale ? __ldg(p.scale + ts.adapter[slot]) : 1.0f;
    uint32_t iter = 0;
    for (int32_t u = cta; u < units; u += p.ctas, ++iter) {
      const int32_t g0 = u / splits * per_group, n = min(per_group, ts.slots - g0);
      if (!warp_wait_inl(bars.acc_full(), iter & 1u, ctl, kSiteAdapterAcc)) break;
      tc_fence_after();
      for (int32_t j = 0; j < n; ++j) {
        const bool mine = slot == g0 + j;
        if (!__any_sync(0xFFFFFFFFu, mine)) continue;
        const uint32_t at = tmem + ((quarter * 32u) << 16) + (uint32_t)(j * p.rank);
        if (splits > 1) {
          // a partial sum: into the ring, rows of rank + 4 values (on different banks)
          const uint32_t dst = ring + (uint32_t)(row * (p.rank + 4)) * 4u;
          for (int32_t c = 0; c < p.rank; c += 8) {
            uint32_t v[8];
            tmem_ld_32x32b_x8(at + (uint32_t)c, v);
            if (mine) {
              st_shared_v4(dst + 4u * (uint32_t)c, v[0], v[1], v[2], v[3]);
              st_shared_v4(dst + 4u * (uint32_t)c + 16u, v[4], v[5], v[6], v[7]);
            }
          }
        } else {
          // the whole sum: its range, then its parts
          RowRange range;
          for (int32_t c = 0; c < p.rank; c += 8) {
            uint32_t v[8];
            tmem_ld_32x32b_x8(at + (uint32_t)c, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) range.add(f * __uint_as_float(v[k]));
          }
          const RowFactor to = row_factor<T>(range, p.f32_out);
          if (mine) {
            p.row_scale[tile * kAdapterRows + row] = to.scale;
            p.row_scale_low[tile * kAdapterRows + row] = to.scale_low;
          }
          bool low = false;
          if constexpr (kWindows) {
            low = __any_sync(0xFFFFFFFFu, mine && to.scale_low != 0.0f);
            if (low) low_mem = 1;
          }
          // (eight zeros past a rank that is not a multiple of the MMA's 16)
          for (int32_t c = 0; c < ((p.rank + 15) & ~15); c += 8) {
            uint32_t v[8] = {};
            if (c < p.rank) tmem_ld_32x32b_x8(at + (uint32_t)c, v);
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = f * __uint_as_float(v[k]);
            T* dst = U + (int64_t)row * pitch + place_of(c);
            if (mine && c < p.rank)
              store_f32<float, 8>(p.u + ((int64_t)tile * kAdapterRows + row) * p.rank + c, o);
            if (mine) store_parts<T, 8, P>(dst, o, to);
            if (low && mine) store_parts<T, 8, P, true>(dst + window, o, to);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.acc_empty());
    }
  }
  tc_fence_before();
  __syncthreads();
  if (splits > 1) {  // the same for the whole cluster: every CTA has one unit or none
    cluster_sync();
    if (cta < units && threadIdx.x < 128) {
      // this CTA's rows of its group, four threads to a row
      const int32_t group = cta / splits, s = cta - group * splits;
      const int32_t r0 = ts.start[group * per_group];
      const int32_t r1 = ts.start[min((group + 1) * per_group, ts.slots)];
      const int32_t quad = (int32_t)threadIdx.x & 3;
      const int32_t rounds = (r1 - r0 + 32 * splits - 1) / (32 * splits);
      for (int32_t k = 0; k < rounds; ++k) {
        const int32_t i = r0 + (k * 32 + ((int32_t)threadIdx.x >> 2)) * splits + s;
        const bool on = i < r1;
        const int32_t row = ts.order[min(i, r1 - 1)];
        const float f = ts.scale[ts.slot[row]];
        const uint32_t src = ring + (uint32_t)(row * (p.rank + 4)) * 4u;
        constexpr int kQuads = kMaxRank / 16;  // of four values, per thread
        float v[kQuads][4];
        RowRange range;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const int32_t c = (q * 4 + quad) * 4;
          v[q][0] = v[q][1] = v[q][2] = v[q][3] = 0.0f;
          if (q * 16 >= p.rank) break;
          if (c < p.rank) {
            // all slices' sums in flight together (one after the other: 5 us for four)
            float4 x[8];
#pragma unroll
            for (int32_t j = 0; j < 8; ++j)
              x[j] = j < splits ? ld_cluster_v4(mapa_shared(src + 4u * (uint32_t)c, (uint32_t)(group * splits + j)))
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int32_t j = 0; j < 8; ++j)
              v[q][0] += x[j].x, v[q][1] += x[j].y, v[q][2] += x[j].z, v[q][3] += x[j].w;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[q][e] *= f;
              range.add(v[q][e]);
            }
            if (on) store_f32<float, 4>(p.u + ((int64_t)tile * kAdapterRows + row) * p.rank + c, v[q]);
          }
        }
        range.join(4);
        const RowFactor to = row_factor<T>(range, p.f32_out);
        if (on && quad == 0) {
          p.row_scale[tile * kAdapterRows + row] = to.scale;
          p.row_scale_low[tile * kAdapterRows + row] = to.scale_low;
        }
        const bool low = kWindows && on && to.scale_low != 0.0f;
        if (low) low_mem = 1;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const int32_t c = (q * 4 + quad) * 4;
          T* dst = U + (int64_t)row * pitch + place_of(c);
          if (on && c < ((p.rank + 15) & ~15)) store_parts<T, 4, P>(dst, v[q], to);
        }
        if (kWindows && __any_sync(0xFFFFFFFFu, low)) {  // (a branch: predicated it cost 3 us)
#pragma unroll
          for (int q = 0; q < kQuads; ++q) {
            const int32_t c = (q * 4 + quad) * 4;
            T* dst = U + (int64_t)row * pitch + window + place_of(c);
            if (low && c < ((p.rank + 15) & ~15)) store_parts<T, 4, P, true>(dst, v[q], to);
          }
        }
      }
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  if (kWindows && threadIdx.x == 0) p.low[tile * kAdaptCtas + cta] = (uint32_t)low_mem;
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, kAdapterCols);
  }
}

template <typename T, int P>
cudaError_t launch(const CUtensorMap& tmX, const CUtensorMap& tmDown, const AdapterParams& p,
                   cudaStream_t stream) {
  auto kernel = adapter_down_kernel<T, P>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = ((int64_t)p.tiles + 1) / 2;
  const int64_t clusters = p.tiles + (pairs + p.ctas - 1) / p.ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * p.ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, tmX, tmDown, p);
}

}  // namespace

cudaError_t launch_adapter_down(const CUtensorMap& tmX, const CUtensorMap& tmDown,
                                const AdapterParams& p, int elem_in, cudaStream_t stream) {
  if (elem_in == kElemF16) return launch<__half, 2>(tmX, tmDown, p, stream);
  return p.parts == 3 ? launch<__nv_bfloat16, 3>(tmX, tmDown, p, stream)
                      : launch<__nv_bfloat16, 2>(tmX, tmDown, p, stream);
}

}  // namespace gb300

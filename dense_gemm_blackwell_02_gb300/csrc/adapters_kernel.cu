// Low-rank adapters beside a shared projection, a different one for every row:
//     Y[i] = W . X[i] + s * Up[a] . (Down[a] . X[i]),   a = row_adapter[i]
// W . X is the GEMM's.  Two kernels add the rest:
//     u[i] = s * Down[a] . X[i]          (adapter_down_kernel, binary32)
//     Y[i] = base[i] + Up[a] . u[i]      (adapter_up_kernel, rounded once)
//
// Both work on tiles of 128 rows in their own order, whatever adapters they name.  A tile's
// distinct adapters are numbered (slots), and the tensor cores multiply the whole tile by
// each of them, every adapter into accumulator columns of its own; a row then takes the
// columns of the one it names.  So rows need no sorting, nothing of one adapter enters
// another row's sums (infinities and NaN included), and the surplus products cost nothing
// that is scarce: the adapters' weights, read once per tile, bound both kernels.
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
}

// Among the four warps that take results out: a barrier, and one that tells whether
// `fail` held in any thread (so that they leave a loop with barriers together).
__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool epilogue_any(bool fail) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p_, q_;\n\tsetp.ne.u32 p_, %1, 0;\n\t"
      "bar.red.or.pred q_, 1, 128, p_;\n\tselp.u32 %0, 1, 0, q_;\n\t}"
      : "=r"(any)
      : "r"(fail ? 1u : 0u)
      : "memory");
  return any != 0;
}

// Where a CTA's barriers stand in shared memory.
struct Bars {
  uint32_t base;
  __device__ uint32_t full(uint32_t s) const { return base + 8u * s; }
  __device__ uint32_t empty(uint32_t s) const { return base + 8u * (kMaxStages + s); }
  __device__ uint32_t acc_full(uint32_t i) const { return base + 8u * (2 * kMaxStages + i); }
  __device__ uint32_t acc_empty(uint32_t i) const { return base + 8u * (2 * kMaxStages + 2 + i); }
  __device__ uint32_t drain() const { return base + 8u * (2 * kMaxStages + 4); }
  __device__ void init() const {
    for (uint32_t s = 0; s < kMaxStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), 4);
    }
    mbar_init(drain(), 1);
    fence_mbarrier_init();
  }
};
constexpr int kNumBars = 2 * kMaxStages + 5;

// ---------------------------------------------------------------------------- Down . X --
// The CTAs of a row tile share its (group of adapters, K slice) units: as many K slices as
// leave every CTA one unit.  A group is what fits 128 accumulator columns.  Slices meet in
// global memory: the last of a group to arrive adds them in slice order.
constexpr uint32_t kDownRing = 96 * 1024;  // two CTAs per SM
constexpr uint32_t kDownSmem = kDownRing + 1024;

__global__ void __launch_bounds__(kThreads, 2)
    adapter_down_kernel(const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmDown, const AdapterParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ TileSlots ts;
  __shared__ alignas(8) uint64_t bar_mem[kNumBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t abort_mem;
  __shared__ int32_t last_mem;
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const Bars bars{smem_addr(bar_mem)};
  const uint32_t warp = warp_id(), lane = lane_id();
  const WaitCtl ctl{p.wait_limit_ns, p.status, &abort_mem};

  if (warp == 0 && lane == 0) {
    bars.init();
    abort_mem = 0;
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

  const int32_t tile = (int32_t)blockIdx.x / p.down_ctas;
  const int32_t cta = (int32_t)blockIdx.x - tile * p.down_ctas;
  number_slots(ts, p, tile * kAdapterRows);
  const int32_t per_group = kAdapterCols / p.rank;
  const int32_t groups = (ts.slots + per_group - 1) / per_group;
  const int32_t splits = groups == 0 ? 1 : min(max(p.down_ctas / groups, 1), p.max_splits);
  const int32_t units = groups * splits;
  // A stage: X's rows, then the group's rows of Down; the MMA's N is a multiple of 16, and
  // it reads 128 rows of X (those past the box only feed rows that nobody takes).
  const uint32_t x_bytes = ((uint32_t)p.x_rows * kRowBytes + 1023u) & ~1023u;
  const uint32_t n_max = ((uint32_t)(min(per_group, ts.slots) * p.rank) + 15u) & ~15u;
  const uint32_t stage_bytes = x_bytes + n_max * kRowBytes;
  const uint32_t reach = max(stage_bytes, kTileBytes);
  const uint32_t stages = min((uint32_t)kMaxStages, 1u + (kDownRing - reach) / max(stage_bytes, 1u));

  if (warp == 0) {
    uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    for (int32_t u = cta; ok && u < units; u += p.down_ctas) {
      const int32_t group = u / splits, s = u - group * splits;
      const int32_t g0 = group * per_group, n = min(per_group, ts.slots - g0);
      const int32_t kb1 = (int32_t)((int64_t)(s + 1) * p.k_blocks / splits);
      for (int32_t kb = (int32_t)((int64_t)s * p.k_blocks / splits); kb < kb1; ++kb) {
        if (!warp_wait_inl(bars.empty(stage), phase ^ 1u, ctl, kSiteAdapterEmpty)) {
          ok = false;
          break;
        }
        const uint32_t at = ring + stage * stage_bytes;
        mbar_arrive_expect_tx_elect(bars.full(stage), (uint32_t)(p.x_rows + n * p.rank) * kRowBytes);
        for (int32_t j = 0; j < n; ++j)
          tma_load_2d_elect(at + x_bytes + (uint32_t)(j * p.rank) * kRowBytes, &tmDown, kb * kBlockK,
                            ts.adapter[g0 + j] * p.rank, bars.full(stage));
        tma_load_2d_elect(at, &tmX, kb * kBlockK, tile * kAdapterRows, bars.full(stage));
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
    for (int32_t u = cta; ok && u < units; u += p.down_ctas, ++iter) {
      const int32_t group = u / splits, s = u - group * splits;
      const int32_t n = min(per_group, ts.slots - group * per_group);
      const uint32_t idesc = p.idesc | ((((uint32_t)(n * p.rank) + 15u) >> 4) << 18);  // N >> 3 at bit 17
      if (!warp_wait_inl(bars.acc_empty(0), (iter & 1u) ^ 1u, ctl, kSiteAdapterAcc)) break;
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
        umma_stage_elect<1>(tmem, smem_desc_sw128_kmajor(at), smem_desc_sw128_kmajor(at + x_bytes),
                            idesc, kb > kb0 ? 1u : 0u, bars.empty(stage));
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      if (ok) umma_commit_elect<1>(bars.acc_full(0));
    }
    // every MMA has read its operands and written its columns before the CTA tears down
    umma_commit_elect<1>(bars.drain());
    if (lane == 0) wait_parity_drain(bars.drain(), 0, ctl);
    __syncwarp();
  } else {
    const uint32_t quarter = warp & 3u;
    const int32_t row = (int32_t)(quarter * 32 + lane);
    const int32_t slot = ts.slot[row];
    const int32_t quads = p.rank / 4;
    uint32_t iter = 0;
    for (int32_t u = cta; u < units; u += p.down_ctas, ++iter) {
      const int32_t group = u / splits, s = u - group * splits;
      const int32_t g0 = group * per_group, n = min(per_group, ts.slots - g0);
      if (epilogue_any(!warp_wait_inl(bars.acc_full(0), iter & 1u, ctl, kSiteAdapterAcc))) break;
      tc_fence_after();
      float* dst = splits == 1
                       ? p.U + (int64_t)(tile * kAdapterRows + row) * p.rank
                       : p.partial + ((int64_t)(tile * p.max_splits + s) * kAdapterRows + row) * p.rank;
      const float f = splits == 1 && slot >= 0 && p.scale ? p.scale[ts.adapter[slot]] : 1.0f;
      for (int32_t j = 0; j < n; ++j) {
        const bool mine = slot == g0 + j;
        if (!__any_sync(0xFFFFFFFFu, mine)) continue;
        for (int32_t c = 0; c < p.rank; c += 8) {
          uint32_t v[8];
          tmem_ld_32x32b_x8(tmem + ((quarter * 32u) << 16) + (uint32_t)(j * p.rank + c), v);
          if (mine) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = f * __uint_as_float(v[k]);
            store_f32<float, 8>(dst + c, o);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.acc_empty(0));
      if (splits == 1) continue;
      // hand the slice over; the last one to arrive adds them all, in order
      __threadfence();
      epilogue_barrier();
      if (threadIdx.x == 64) {
        uint32_t* ctr = p.counters + tile * kAdapterRows + group;
        const uint32_t old = atom_add_acq_rel_gpu(ctr, 1u);
        last_mem = old == (uint32_t)splits - 1u;
        if (last_mem) st_relaxed_gpu_u32(ctr, 0u);
      }
      epilogue_barrier();
      if (last_mem) {
        __threadfence();
        const int32_t r0 = ts.start[g0], count = (ts.start[g0 + n] - r0) * quads;
        const float* part = p.partial + (int64_t)tile * p.max_splits * kAdapterRows * p.rank;
        const int64_t pitch = (int64_t)kAdapterRows * p.rank;
        for (int32_t i = (int32_t)threadIdx.x - 64; i < count; i += 128) {
          const int32_t r = ts.order[r0 + i / quads], c = (i % quads) * 4;
          const float* src = part + (int64_t)r * p.rank + c;
          float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int32_t k = 0; k < splits; k += 8) {
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              v[q] = k + q < splits ? ld_global_cg_v4(src + (k + q) * pitch) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (k + q < splits) {
                sum.x += __uint_as_float(v[q].x);
                sum.y += __uint_as_float(v[q].y);
                sum.z += __uint_as_float(v[q].z);
                sum.w += __uint_as_float(v[q].w);
              }
          }
          const float f2 = p.scale ? p.scale[ts.id[r]] : 1.0f;
          *reinterpret_cast<float4*>(p.U + (int64_t)(tile * kAdapterRows + r) * p.rank + c) =
              make_float4(f2 * sum.x, f2 * sum.y, f2 * sum.z, f2 * sum.w);
        }
      }
      epilogue_barrier();  // last_mem may change
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, kAdapterCols);
  }
}

// ------------------------------------------------------------------------------ Up . u --
// The CTAs of a row tile share Y's column tiles.  The tile's u is the row operand of every
// product: it is split into two 16-bit parts, u = 2^e (hi + lo) with e the exponent of the
// row's largest value, so that fp16's range cannot cut it off and at least 17 of its bits
// reach the product (one part alone would round u to 8 or 11 bits, an error of the size of
// Y's own rounding).  A column tile times a slot's adapter lands in one of two accumulators.
constexpr uint32_t kUpRing2 = 4;  // stages with ranks up to 64; 2 above

__host__ __device__ constexpr uint32_t up_stages(int rank) { return rank <= 64 ? kUpRing2 : 2; }
__host__ __device__ constexpr uint32_t up_smem(int rank) {
  return (rank <= 64 ? 2u : 4u) * kTileBytes + up_stages(rank) * kTileBytes + 1024u;
}

template <typename T, typename TO, bool BASE>
__global__ void __launch_bounds__(kThreads, 2)
    adapter_up_kernel(const __grid_constant__ CUtensorMap tmUp, const AdapterParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ TileSlots ts;
  __shared__ alignas(8) uint64_t bar_mem[kNumBars];
  __shared__ float row_scale[kAdapterRows];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t abort_mem;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int32_t chunks = p.rank <= 64 ? 1 : 2;
  const uint32_t ring = base + 2u * (uint32_t)chunks * kTileBytes;
  const uint32_t stages = up_stages(p.rank);
  const Bars bars{smem_addr(bar_mem)};
  const uint32_t warp = warp_id(), lane = lane_id();
  const WaitCtl ctl{p.wait_limit_ns, p.status, &abort_mem};

  if (warp == 0 && lane == 0) {
    bars.init();
    abort_mem = 0;
    tma_prefetch_desc(&tmUp);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_addr(&tmem_slot), 2 * kAdapterCols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  const int32_t tile = (int32_t)blockIdx.x / p.up_ctas;
  const int32_t cta = (int32_t)blockIdx.x - tile * p.up_ctas;
  const int32_t n_tiles = (p.N + kAdapterCols - 1) / kAdapterCols;
  number_slots(ts, p, tile * kAdapterRows);

  // u -> the row operand: part (2 * chunk + lo) is a 128 x 64 tile in the 128-byte swizzle
  if (threadIdx.x < kAdapterRows) {
    const int32_t row = (int32_t)threadIdx.x;
    const bool any = ts.slot[row] >= 0;
    const float* u = p.U + (int64_t)(tile * kAdapterRows + row) * p.rank;
    float big = 0.0f;
    if (any)
      for (int32_t c = 0; c < p.rank; c += 8) {
        float v[8];
        load_f32<float, 8>(u + c, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(v[k]));
      }
    // 2^e and its inverse from the exponent field; 1 for zero and for infinities (NaN is
    // not counted by fmaxf and passes through any scaling)
    int32_t e = (int32_t)(__float_as_uint(big) >> 23);
    if (e == 0 || e == 255) e = 127;
    e = min(max(e, 2), 252);
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    row_scale[row] = __uint_as_float((uint32_t)e << 23);
    for (int32_t c = 0; c < 64 * chunks; c += 8) {
      Pack<T, 8> hi, lo;
      float v[8] = {};
      if (any && c < p.rank) load_f32<float, 8>(u + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = v[k] * inv;
        hi.v[k] = from_f32<T>(x);
        const float h = to_f32(hi.v[k]);
        lo.v[k] = from_f32<T>(isinf(h) ? 0.0f : x - h);
      }
      const uint32_t at = base + (uint32_t)(c >> 6) * 2u * kTileBytes + (uint32_t)row * kRowBytes +
                          ((((uint32_t)c >> 3) & 7u) ^ ((uint32_t)row & 7u)) * 16u;
      const uint4 h4 = *reinterpret_cast<const uint4*>(&hi), l4 = *reinterpret_cast<const uint4*>(&lo);
      st_shared_v4(at, h4.x, h4.y, h4.z, h4.w);
      st_shared_v4(at + kTileBytes, l4.x, l4.y, l4.z, l4.w);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();

  if (warp == 0) {
    uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    for (int32_t j = cta; ok && j < n_tiles; j += p.up_ctas)
      for (int32_t d = 0; ok && d < ts.slots; ++d)
        for (int32_t c = 0; c < chunks; ++c) {
          if (!warp_wait_inl(bars.empty(stage), phase ^ 1u, ctl, kSiteAdapterEmpty)) {
            ok = false;
            break;
          }
          // (the last tile's rows past N are the next adapter's: columns that are not stored)
          mbar_arrive_expect_tx_elect(bars.full(stage), kTileBytes);
          tma_load_2d_elect(ring + stage * kTileBytes, &tmUp, c * kBlockK,
                            ts.adapter[d] * p.N + j * kAdapterCols, bars.full(stage));
          armed |= 1u << stage;
          armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
    if (lane == 0)
      for (uint32_t s = 0; s < stages; ++s)
        if (armed & (1u << s)) wait_parity_drain(bars.full(s), (armed_phase >> s) & 1u, ctl);
    __syncwarp();
  } else if (warp == 1) {
    uint32_t stage = 0, phase = 0, iter = 0;
    bool ok = true;
    const uint32_t idesc = p.idesc | ((uint32_t)(kAdapterCols >> 3) << 17);
    for (int32_t j = cta; ok && j < n_tiles; j += p.up_ctas)
      for (int32_t d = 0; ok && d < ts.slots; ++d, ++iter) {
        const uint32_t slot = iter & 1u;
        if (!warp_wait_inl(bars.acc_empty(slot), ((iter >> 1) & 1u) ^ 1u, ctl, kSiteAdapterAcc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int32_t c = 0; c < chunks; ++c) {
          if (!warp_wait_inl(bars.full(stage), phase, ctl, kSiteAdapterFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b = smem_desc_sw128_kmajor(ring + stage * kTileBytes);
          const int32_t steps = (min(p.rank - 64 * c, 64) + 15) / 16;
          for (int32_t part = 0; part < 2; ++part) {
            const uint64_t a = smem_desc_sw128_kmajor(base + (uint32_t)(2 * c + part) * kTileBytes);
            for (int32_t k = 0; k < steps; ++k)  // 16 values: 32 bytes, 2 in the descriptor
              umma_f16_elect(tmem + slot * kAdapterCols, a + 2u * (uint32_t)k, b + 2u * (uint32_t)k,
                             idesc, (c | part | k) ? 1u : 0u);
          }
          umma_commit_elect<1>(bars.empty(stage));
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
        if (ok) umma_commit_elect<1>(bars.acc_full(slot));
      }
    umma_commit_elect<1>(bars.drain());
    if (lane == 0) wait_parity_drain(bars.drain(), 0, ctl);
    __syncwarp();
  } else {
    const uint32_t quarter = warp & 3u;
    const int32_t row = (int32_t)(quarter * 32 + lane);
    const int64_t i = (int64_t)tile * kAdapterRows + row;
    const int32_t slot = ts.slot[row];
    const bool live = i < p.M;
    const float rs = row_scale[row];
    uint32_t iter = 0;
    // one piece of 32 columns of this thread's row: base + rs * v
    auto write = [&](int32_t n0, const uint32_t (&v)[32]) {
      TO* y = static_cast<TO*>(p.Y) + i * p.N + n0;
      const float* b = BASE ? p.base + i * p.N + n0 : nullptr;
      constexpr int V = 16 / (int)sizeof(TO);
      if (p.vec_store && n0 + 32 <= p.N) {
#pragma unroll
        for (int c = 0; c < 32; c += V) {
          float o[V];
          if constexpr (BASE) {
            load_f32<float, V>(b + c, o);
          } else {
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = 0.0f;
          }
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = fmaf(rs, __uint_as_float(v[c + k]), o[k]);
          store_f32<TO, V>(y + c, o);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (n0 + c < p.N) y[c] = from_f32<TO>(fmaf(rs, __uint_as_float(v[c]), BASE ? b[c] : 0.0f));
      }
    };
    bool ok = true;
    for (int32_t j = cta; ok && j < n_tiles; j += p.up_ctas) {
      const int32_t n0 = j * kAdapterCols;
      // rows without an adapter: the base alone (in place already there), or zero
      if (live && slot < 0 && !(BASE && static_cast<const void*>(p.base) == p.Y)) {
        const uint32_t zero[32] = {};
        for (int32_t c = 0; c < kAdapterCols; c += 32) write(n0 + c, zero);
      }
      for (int32_t d = 0; d < ts.slots; ++d, ++iter) {
        const uint32_t acc = iter & 1u;
        if (!warp_wait_inl(bars.acc_full(acc), (iter >> 1) & 1u, ctl, kSiteAdapterAcc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool mine = live && slot == d;
        if (__any_sync(0xFFFFFFFFu, mine)) {
          for (int32_t c = 0; c < kAdapterCols; c += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tmem + ((quarter * 32u) << 16) + acc * kAdapterCols + (uint32_t)c, v);
            tmem_ld_wait(v);
            if (mine) write(n0 + c, v);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.acc_empty(acc));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 2 * kAdapterCols);
  }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int64_t grid, uint32_t smem, cudaStream_t stream,
                   const Args&... args) {
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, typename TO>
cudaError_t up_by_base(const CUtensorMap& tmUp, const AdapterParams& p, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.tiles * p.up_ctas;
  return p.base ? launch(adapter_up_kernel<T, TO, true>, grid, up_smem(p.rank), stream, tmUp, p)
                : launch(adapter_up_kernel<T, TO, false>, grid, up_smem(p.rank), stream, tmUp, p);
}

template <typename T>
cudaError_t up_by_out(const CUtensorMap& tmUp, const AdapterParams& p, int elem_out,
                      cudaStream_t stream) {
  switch (elem_out) {
    case kElemF16: return up_by_base<T, __half>(tmUp, p, stream);
    case kElemBF16: return up_by_base<T, __nv_bfloat16>(tmUp, p, stream);
    case kElemF32: return up_by_base<T, float>(tmUp, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_adapter_down(const CUtensorMap& tmX, const CUtensorMap& tmDown,
                                const AdapterParams& p, cudaStream_t stream) {
  return launch(adapter_down_kernel, (int64_t)p.tiles * p.down_ctas, kDownSmem, stream, tmX, tmDown, p);
}

cudaError_t launch_adapter_up(const CUtensorMap& tmUp, const AdapterParams& p, int elem_in,
                              int elem_out, cudaStream_t stream) {
  if (elem_in == kElemF16) return up_by_out<__half>(tmUp, p, elem_out, stream);
  return up_by_out<__nv_bfloat16>(tmUp, p, elem_out, stream);
}

}  // namespace gb300

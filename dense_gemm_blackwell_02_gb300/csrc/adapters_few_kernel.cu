// Low-rank adapters for a batch of few rows (decoding: a row per request), beside the shared
// product W . x that the GEMM leaves in `base`:
//     u[i] = s * Down[a] . x[i]            (few_down_kernel, partial sums)
//     Y[i] = base[i] + Up[a] . u[i]        (few_up_kernel, rounded once)
//
// Every adapter's weights are read once for at most 16 rows: 2 rank (K + N) values against
// some tens of rows, so HBM and latency bound it, and the 16-row warp MMA (m16n8k16) is the
// shape that wastes nothing; a 128-row tcgen05 tile would be filled to a tenth.
//
// The rows that name one adapter form groups of 16.  few_down runs beside the GEMM: it is
// launched after it but waits for it only at its end (programmatic dependent launch; what
// it reads are the call's inputs, complete when the GEMM started).  Next to a CTA of the
// GEMM an SM has room for one of few_down's (80 registers for 128 threads, 5 KiB of shared
// memory where the GEMM keeps its staging in the ring), alone for six, so the GEMM's tiling
// leaves it some SMs.  A CTA's warps share a K slice of 16 values of a group's u, weights
// straight from global memory into MMA fragments, and leave partial sums for few_up to add
// in order.  Ahead of the GEMM instead of beside it the whole is slower (64 adapters of
// rank 16, 256 x 10240 x 8192 67 us against 55; 256 x 1000 x 2048 32 against 15).
//
// Measured, bf16 over cold operands, 256 x 10240 x 8192, 64 adapters of rank 16: 56 us, of
// which the product alone is 40 (168 MB, 4.2 TB/s) and few_up after it 10 (Up's 21 MB from
// HBM, the binary32 product's 10 MB from L2); few_down's 17 MB cost the product 5.  One row,
// 8192 x 8192: 30 us, the product alone 26.  Binary32 results take a third part of u: 58 to 60
// us for the first.  Looking further ahead in few_up spills and costs 2 us; Up brought into L2
// during the product gains nothing.
//
// A dot product does not care in which order K is taken: lane t of a fragment's four reads
// eight consecutive values, in both operands alike, where the fragment's layout would give
// it four pairs; likewise the columns of four 8-column tiles are dealt so that a lane ends
// up with eight neighbouring columns of Y.
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = kFewGroup;   // rows of one adapter that are taken together
constexpr int kUnitRank = 16;      // values of u per unit of few_down
constexpr int kMaxChecks = 8;      // rows that a CTA of few_down looks at, at most

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 values of K: two MMAs on 16-byte chunks of rows g and g + 8 and of a column.
template <typename T>
__device__ __forceinline__ void mma32(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& b) {
  mma16816<T>(d, x0.x, x1.x, x0.y, x1.y, b.x, b.y);
  mma16816<T>(d, x0.z, x1.z, x0.w, x1.w, b.z, b.w);
}

// The adapter of row i: -1 for none or an id past the pool, -2 past the batch.
__device__ __forceinline__ int32_t adapter_of(const AdapterFewParams& p, int32_t i) {
  if (i >= p.M) return -2;
  const int32_t a = __ldg(p.row_adapter + i);
  return a < 0 || a >= p.count ? -1 : a;
}

// Whether row i begins a group: 16, 32, ... (or no) rows before it name its adapter.
__device__ __forceinline__ bool begins_group(const AdapterFewParams& p, int row) {
  const int32_t a = adapter_of(p, row);
  int before = 0;
  for (int j = (int)lane_id(); j < row; j += 32) before += adapter_of(p, j) == a;
  return __reduce_add_sync(0xFFFFFFFFu, before) % kRows == 0;
}

template <typename T>
__device__ __forceinline__ void few_down_unit(const AdapterFewParams& p, int row, bool lists) {
  const int warp = (int)warp_id(), lane = (int)lane_id();
  const int32_t a = adapter_of(p, row);
  // lane r of 16: the group's r-th row
  int mine = -1;
  for (int j0 = row & ~31, n = 0; j0 < p.M && n < kRows; j0 += 32) {
    uint32_t m = __ballot_sync(0xFFFFFFFFu, j0 + lane >= row && adapter_of(p, j0 + lane) == a);
    for (; m != 0 && n < kRows; m &= m - 1, ++n)
      if (lane == n) mine = j0 + __ffs((int)m) - 1;
  }
  if (lists) {
    int at = lane == 0 ? (int)atomicAdd(p.counts, 1u) : 0;
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, mine >= 0));
    if ((uint32_t)at < (uint32_t)p.M) {  // (always, as long as the counter began at zero)
      FewGroup& entry = p.groups[at];
      if (lane < kRows) entry.row[lane] = mine;
      if (lane == 0) entry.adapter = a, entry.rows = n;
    }
  }
  if (a < 0) return;
  const int g = lane >> 2, t = lane & 3;
  const int row0 = __shfl_sync(0xFFFFFFFFu, mine, g), row1 = __shfl_sync(0xFFFFFFFFu, mine, g + 8);
  __shared__ int16_t rows_mem[kRows];
  if (warp == 0 && lane < kRows) rows_mem[lane] = (int16_t)mine;
  const int live = __popc(__ballot_sync(0xFFFFFFFFu, mine >= 0));
  const int slice = (int)blockIdx.z * kWarps + warp, slices = p.slices * kWarps;
  const int r = (int)blockIdx.y * kUnitRank;

  constexpr int kSteps = 3;  // of 32 values of K, whose loads are in flight together
  const T* x0 = static_cast<const T*>(p.X) + (int64_t)max(row0, 0) * p.K;
  const T* x1 = static_cast<const T*>(p.X) + (int64_t)max(row1, 0) * p.K;
  const T* d0 = static_cast<const T*>(p.down) + ((int64_t)a * p.rank + r + g) * p.K;
  const T* d1 = d0 + (int64_t)8 * p.K;
  const bool second = r + 8 < p.rank;
  float acc[2][4] = {};
  // the slices are interleaved step by step, so that warps side by side read side by side
  for (int k0 = slice * 32 + 8 * t; k0 - 8 * t < p.K; k0 += kSteps * slices * 32) {
    uint4 xa[kSteps], xb[kSteps], b0[kSteps], b1[kSteps];
    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const int k = k0 + q * slices * 32;
      const bool in = k < p.K;
      b0[q] = in ? ldg_stream(d0 + k) : z;
      b1[q] = in && second ? ldg_stream(d1 + k) : z;
      xa[q] = in && row0 >= 0 ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : z;
      xb[q] = in && row1 >= 0 ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : z;
    }
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      mma32<T>(acc[0], xa[q], xb[q], b0[q]);
      mma32<T>(acc[1], xa[q], xb[q], b1[q]);
    }
  }
  // the CTA's four slices are added here: partial[row][slice][rank]
  __shared__ float red[kWarps][kRows][kUnitRank + 2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    *reinterpret_cast<float2*>(&red[warp][g][8 * j + 2 * t]) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(&red[warp][g + 8][8 * j + 2 * t]) = make_float2(acc[j][2], acc[j][3]);
  }
  __syncthreads();
  for (int e = (int)threadIdx.x; e < live * kUnitRank; e += kThreads) {
    const int i = e / kUnitRank, c = e % kUnitRank;
    if (r + c >= p.rank) continue;
    float sum = red[0][i][c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += red[w][i][c];
    const int at = (int)rows_mem[i];
    p.partial[((int64_t)at * p.slices + (int)blockIdx.z) * p.rank + r + c] = sum;
  }
}

// A unit: the group that a row begins (if it begins one), 16 values of u, one CTA's share
// of K.  Grid: x the rows, y the 16 values, z the CTAs' shares.  A CTA looks at `checks`
// rows, one per warp at a time, because a CTA that only finds that its row begins nothing
// still costs its launch; the rows are dealt so that neither the first rows of a mixed
// batch, which all begin groups, nor every 16th of a sorted one fall to the same CTAs.
// The groups are listed in the order in which the atomic counter
// numbers them, which nothing but few_up's schedule depends on.
template <typename T, bool ALONE>
__global__ void __launch_bounds__(kThreads, 6) few_down_kernel(const AdapterFewParams p) {
  const int warp = (int)warp_id(), lane = (int)lane_id();
  const bool lists = blockIdx.y == 0 && blockIdx.z == 0;
  const auto check = [&](int row, bool reports) {
    if (reports && lane == 0 && __ldg(p.row_adapter + row) >= p.count)
      record_bad_index(p.status, kSiteRowAdapter);
    return begins_group(p, row);
  };
  if constexpr (ALONE) {  // checks == 1: every warp looks at it, without a barrier
    const int row = (int)blockIdx.x;
    if (check(row, lists && warp == 0)) few_down_unit<T>(p, row, lists && warp == 0);
  } else {
    const auto row_of = [](int c) {
      return c * (int)gridDim.x + ((int)blockIdx.x + 3 * c) % (int)gridDim.x;
    };
    __shared__ uint32_t found[kWarps];
    uint32_t begins = 0;  // bit c: row_of(c) begins a group
    for (int c = warp; c < p.checks; c += kWarps)
      if (row_of(c) < p.M && check(row_of(c), lists)) begins |= 1u << c;
    if (lane == 0) found[warp] = begins;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) begins |= found[w];
    for (; begins != 0; begins &= begins - 1) {
      few_down_unit<T>(p, row_of(__ffs((int)begins) - 1), lists && warp == 0);
      __syncthreads();  // (the next unit writes the same shared memory)
    }
  }
  // This grid counts as complete only after the GEMM, so that those after it wait for both.
  if (blockIdx.x == 0 && lists && warp == 0) grid_dependency_wait();
}

// 8 or 16 bytes of a row: four or eight values.
template <int RC> struct Chunk { using type = uint4; static constexpr int kValues = 8; };
template <> struct Chunk<16> { using type = uint2; static constexpr int kValues = 4; };

template <typename T>
__device__ __forceinline__ void mma_chunk(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& b) {
  mma32<T>(d, x0, x1, b);
}
template <typename T>
__device__ __forceinline__ void mma_chunk(float (&d)[4], const uint2& x0, const uint2& x1, const uint2& b) {
  mma16816<T>(d, x0.x, x1.x, x0.y, x1.y, b.x, b.y);
}
__device__ __forceinline__ void ldg_chunk(uint4& v, const void* p) { v = ldg_stream(p); }
__device__ __forceinline__ void ldg_chunk(uint2& v, const void* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
}

// The parts of neighbouring values of a row's second window: of those below `least`, divided by
// the window's factor (0: the row has none).
template <typename T, int P, typename C>
__device__ __forceinline__ void low_parts(const float* u, float least, float factor, C (&part)[P]) {
  constexpr int N = sizeof(C) / sizeof(T);
  const float inv = factor != 0.0f ? 1.0f / factor : 0.0f;
  Pack<T, N> to[P];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    T x[P];
    split_f32(factor != 0.0f && fabsf(u[k]) < least ? u[k] * inv : 0.0f, x);
#pragma unroll
    for (int j = 0; j < P; ++j) to[j].v[k] = x[j];
  }
#pragma unroll
  for (int j = 0; j < P; ++j) memcpy(&part[j], &to[j], sizeof(C));
}

__host__ __device__ constexpr int up_ctas_per_sm(int rc) { return rc <= 16 ? 6 : rc <= 32 ? 5 : 4; }

// Grid: x a share of Y's columns, y the group.  RC: the rank's class, 16, 32, 64 or 128.  A
// warp takes 32 columns at a time, and loads the next ones' weights and base before it
// multiplies the present ones'.  u enters the MMA as 16-bit parts (RowFactor, split_f32).
template <typename T, typename TO, int RC>
__global__ void __launch_bounds__(kThreads, up_ctas_per_sm(RC))
    few_up_kernel(const __grid_constant__ AdapterFewParams p) {
  using C = typename Chunk<RC>::type;
  constexpr int kValues = Chunk<RC>::kValues;       // of a row per lane and chunk
  constexpr int kChunks = RC / (4 * kValues);       // chunks of a row
  constexpr int kPitch = RC + 8;  // values per row of a part: rows on different banks
  constexpr int P = u_parts(std::is_same<T, __nv_bfloat16>::value, std::is_same<TO, float>::value);
  __shared__ alignas(16) T part[P][kRows * kPitch];
  __shared__ float row_scale[kRows], row_scale_low[kRows];  // (RowFactor)
  __shared__ alignas(16) float u_mem[kRows][RC + 4];
  __shared__ float turn[kWarps][8][33];
  const int tid = (int)threadIdx.x, warp = (int)warp_id(), lane = (int)lane_id();
  const int g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t total = __ldcg(p.counts);
  const FewGroup* entry = p.groups + blockIdx.y;
  const int32_t a = __ldcg(&entry->adapter), live = __ldcg(&entry->rows);
  const int row0 = __ldcg(entry->row + g), row1 = __ldcg(entry->row + g + 8);
  constexpr int kLanes = RC / 8;            // threads per row of u, eight values each
  constexpr int kPass = kThreads / kLanes;  // rows at a time
  const int my_row = __ldcg(entry->row + min(tid / kLanes, kRows - 1));
  const bool in_place = static_cast<const void*>(p.base) == p.Y;

  if (blockIdx.y < total && !(a < 0 && in_place)) {
    const int groups = (p.N + 31) / 32;
    const int stride = (int)gridDim.x * kWarps;
    int q = (int)blockIdx.x * kWarps + warp;
    C b[kChunks][4];
    float o[8];
    const T* up = static_cast<const T*>(p.up) + (int64_t)max(a, 0) * p.N * p.rank;
    auto load_up = [&](int qq, C (&dst)[kChunks][4]) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = qq * 32 + 8 * (g >> 1) + 2 * j + (g & 1), k = (4 * c + t) * kValues;
          dst[c][j] = C{};
          if (a >= 0 && n < p.N && k < p.rank) ldg_chunk(dst[c][j], up + (int64_t)n * p.rank + k);
        }
    };
    auto load_base = [&](int qq, int row, float (&dst)[8]) {
      const int n = qq * 32 + 8 * t;
      const float* src = p.base + (int64_t)max(row, 0) * p.base_pitch + n;
#pragma unroll
      for (int k = 0; k < 8; ++k) dst[k] = 0.0f;
      if (row < 0 || qq >= groups) return;
      if (p.vec_base && n + 8 <= p.N) {
        const uint4 x = ld_global_cg_v4(src), y = ld_global_cg_v4(src + 4);
        dst[0] = __uint_as_float(x.x), dst[1] = __uint_as_float(x.y);
        dst[2] = __uint_as_float(x.z), dst[3] = __uint_as_float(x.w);
        dst[4] = __uint_as_float(y.x), dst[5] = __uint_as_float(y.y);
        dst[6] = __uint_as_float(y.z), dst[7] = __uint_as_float(y.w);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (n + k < p.N) dst[k] = __ldcg(src + k);
      }
    };
    auto store = [&](int qq, int row, const float (&src)[8]) {
      const int n = qq * 32 + 8 * t;
      TO* y = static_cast<TO*>(p.Y);
      if (p.vec_store) {
        if (row >= 0 && n < p.N) store_f32<TO, 8>(y + (int64_t)row * p.N + n, src);
        return;
      }
      // Y's rows begin anywhere: through shared memory, so that a store of the warp writes
      // 32 neighbouring values of a row rather than one of eight rows' every eighth
#pragma unroll
      for (int k = 0; k < 8; ++k) turn[warp][g][8 * t + k] = src[k];
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int to = __shfl_sync(0xFFFFFFFFu, row, 4 * r);
        if (to >= 0 && qq * 32 + lane < p.N)
          y[(int64_t)to * p.N + qq * 32 + lane] = from_f32<TO>(turn[warp][r][lane]);
      }
      __syncwarp();
    };
    load_up(q, b);
    load_base(q, row0, o);

    if (a >= 0) {
      const float scale = p.scale ? __ldg(p.scale + a) : 1.0f;
#pragma unroll
      for (int i0 = 0; i0 < kRows; i0 += kPass) {
        const int i = i0 + tid / kLanes, c = tid % kLanes * 8;
        const int row = i >= kRows ? -1 : i0 == 0 ? my_row : __ldcg(entry->row + i);
        float v[8] = {};
        if (row >= 0 && c < p.rank) {
          const float* src = p.partial + (int64_t)row * p.slices * p.rank + c;
          for (int s0 = 0; s0 < p.slices; s0 += 4) {
            uint4 w[4][2];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const float* f = src + (int64_t)(s0 + s) * p.rank;
              const uint4 z = make_uint4(0, 0, 0, 0);
              w[s][0] = s0 + s < p.slices ? ld_global_cg_v4(f) : z;
              w[s][1] = s0 + s < p.slices ? ld_global_cg_v4(f + 4) : z;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint32_t x[8] = {w[s][0].x, w[s][0].y, w[s][0].z, w[s][0].w,
                                     w[s][1].x, w[s][1].y, w[s][1].z, w[s][1].w};
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] += __uint_as_float(x[k]);
            }
          }
        }
        RowRange range;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] *= scale;
          range.add(v[k]);
        }
        range.join(kLanes);
        const RowFactor to = row_factor<T>(range, std::is_same<TO, float>::value);
        if (i < kRows) {
          if (c == 0) row_scale[i] = to.scale, row_scale_low[i] = to.scale_low;
          store_f32<float, 8>(&u_mem[i][c], v);
          Pack<T, 8> x8[P];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            T x[P];
            // (a row with a NaN has NaN for its factor; its parts need not make more of them)
            split_f32(isnan(to.scale) ? 0.0f : to.high(v[k]), x);
#pragma unroll
            for (int j = 0; j < P; ++j) x8[j].v[k] = x[j];
          }
#pragma unroll
          for (int j = 0; j < P; ++j) *reinterpret_cast<Pack<T, 8>*>(part[j] + i * kPitch + c) = x8[j];
        }
      }
      __syncthreads();
    }
    const float s0 = a >= 0 ? row_scale[g] : 0.0f, s1 = a >= 0 ? row_scale[g + 8] : 0.0f;

    auto multiply = [&](const C (&w)[kChunks][4], float (&acc)[4][4]) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int k = (4 * c + t) * kValues;
        C u0[P], u1[P];
#pragma unroll
        for (int s = 0; s < P; ++s) {
          u0[s] = *reinterpret_cast<const C*>(part[s] + g * kPitch + k);
          u1[s] = *reinterpret_cast<const C*>(part[s] + (g + 8) * kPitch + k);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int s = 0; s < P; ++s) mma_chunk<T>(acc[j], u0[s], u1[s], w[c][j]);
      }
    };
    // Whether a lane's columns of a row (first 0: row g, 2: row g + 8) hold an infinity or a NaN,
    // which times zero is NaN; all four lanes' of the row where store() writes for all of them.
    // (Votes in the loop make each step wait for its products: 1 us of the kernel's 10, 3 of 22
    // with rank 64.)
    auto left_out = [&](const float (&acc)[4][4], int first) {
      float z0 = 0.0f, z1 = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) fma2_rn(z0, z1, acc[j][first], acc[j][first + 1], 0.0f);
      bool out = z0 + z1 != 0.0f;
      if (!p.vec_store) out = ((__ballot_sync(0xFFFFFFFFu, out) >> (lane & ~3)) & 0xFu) != 0;
      return out;
    };
    // One of the rows has a second window, or is not held by its parts: its columns are all left
    // to the second pass.
    const float low0 = a >= 0 ? row_scale_low[g] : 0.0f, low1 = a >= 0 ? row_scale_low[g + 8] : 0.0f;
    const bool wide = __any_sync(0xFFFFFFFFu, s0 < 0.0f || s1 < 0.0f || low0 != 0.0f || low1 != 0.0f) != 0;
    bool again = wide;
    for (; !wide && q < groups; q += stride) {
      C bn[kChunks][4];
      float on[8];
      constexpr bool kAhead = RC <= 64;  // (128 values of a row twice do not fit the registers)
      if constexpr (kAhead) {
        if (q + stride < groups) {
          load_up(q + stride, bn);
          load_base(q + stride, row0, on);
        }
      }
      float acc[4][4] = {};
      if (a >= 0) multiply(b, acc);
      const bool out0 = left_out(acc, 0), out1 = left_out(acc, 2);
      again |= out0 || out1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[2 * j] = fmaf(s0, acc[j][0], o[2 * j]);
        o[2 * j + 1] = fmaf(s0, acc[j][1], o[2 * j + 1]);
      }
      store(q, out0 ? -1 : row0, o);
      if (live > 8) {  // rows 8..15 of the group
        load_base(q, row1, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[2 * j] = fmaf(s1, acc[j][2], o[2 * j]);
          o[2 * j + 1] = fmaf(s1, acc[j][3], o[2 * j + 1]);
        }
        store(q, out1 ? -1 : row1, o);
      }
      if (q + stride < groups) {
        if constexpr (kAhead) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) b[c][j] = bn[c][j];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = on[k];
        } else {
          load_up(q + stride, b);
          load_base(q + stride, row0, o);
        }
      }
    }
    // The columns left out: rows with a second window, those that the parts do not hold, and what
    // is not finite, the last two in binary32.
    if (__any_sync(0xFFFFFFFFu, again)) {
      const bool lows = __any_sync(0xFFFFFFFFu, low0 != 0.0f || low1 != 0.0f) != 0;
      for (q = (int)blockIdx.x * kWarps + warp; q < groups; q += stride) {
        load_up(q, b);
        float acc[4][4] = {}, acc_low[4][4] = {};
        multiply(b, acc);
        if constexpr (std::is_same<T, __half>::value) {
          if (lows) {  // (the second window's parts: from u, at every step)
            constexpr float kLeast = window_least(std::is_same<TO, float>::value);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int k = (4 * c + t) * kValues;
              C u0[P], u1[P];
              low_parts<T, P>(&u_mem[g][k], kLeast * s0, low0, u0);
              low_parts<T, P>(&u_mem[g + 8][k], kLeast * s1, low1, u1);
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < P; ++s) mma_chunk<T>(acc_low[j], u0[s], u1[s], b[c][j]);
            }
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool out = wide || left_out(acc, 2 * half);
          const int row = !out ? -1 : half ? row1 : row0;
          const float s = half ? s1 : s0, low = half ? low1 : low0;
          load_base(q, row, o);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x = acc[k / 2][2 * half + k % 2];
            const int n = min(q * 32 + 8 * t + k, p.N - 1);
            if (s < 0.0f || (s > 0.0f && !(fabsf(x) < __builtin_huge_valf()))) {
              o[k] += up_times_u(up + (int64_t)n * p.rank, u_mem[g + 8 * half], p.rank);
            } else {
              o[k] = fmaf(s, x, o[k]);
              if (low != 0.0f) o[k] = fmaf(low, acc_low[k / 2][2 * half + k % 2], o[k]);
            }
          }
          store(q, row, o);
        }
      }
    }
  }
  // the last CTA to have read the list's length clears it for the next call
  __syncthreads();
  if (tid == 0 && atomicAdd(p.counts + 1, 1u) == gridDim.x * gridDim.y - 1u) p.counts[0] = p.counts[1] = 0;
}

cudaError_t launch(void (*kernel)(AdapterFewParams), dim3 grid, const AdapterFewParams& p,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int rank_class(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

template <typename T, typename TO>
void (*up_by_rank(int rank))(AdapterFewParams) {
  switch (rank_class(rank)) {
    case 16: return few_up_kernel<T, TO, 16>;
    case 32: return few_up_kernel<T, TO, 32>;
    case 64: return few_up_kernel<T, TO, 64>;
    default: return few_up_kernel<T, TO, 128>;
  }
}

template <typename T>
void (*up_kernel(int rank, int elem_out))(AdapterFewParams) {
  return elem_out == kElemF16 ? up_by_rank<T, __half>(rank)
                              : elem_out == kElemBF16 ? up_by_rank<T, __nv_bfloat16>(rank) : up_by_rank<T, float>(rank);
}

// Groups there can be at most: one per adapter in use (and one of the rows without), and one
// more for every 16 rows.
int64_t max_groups(const AdapterFewParams& p) {
  return std::min<int64_t>(p.M, std::min<int64_t>(p.M, (int64_t)p.count + 1) + p.M / kRows);
}

}  // namespace

int64_t few_down_rows(int32_t M, int32_t rank, int32_t count) {
  AdapterFewParams p = {};
  p.M = M;
  p.count = count;
  return max_groups(p) * ((rank + kUnitRank - 1) / kUnitRank * kUnitRank);
}

int few_slices(int32_t M, int32_t K, int32_t rank, int32_t count, int sms) {
  // As many K slices as give every SM its six CTAs, a warp at least four steps of 32.
  const int64_t units = few_down_rows(M, rank, count) / kUnitRank;
  const int64_t steps = ((int64_t)K + 31) / 32;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)6 * sms / units, steps / (4 * kWarps), 16}));
}

cudaError_t launch_adapter_few(AdapterFewParams p, int elem_in, int elem_out, int sms,
                               cudaStream_t stream) {
  const bool f16 = elem_in == kElemF16;
  // (half as many units as CTAs, so that few CTAs find two)
  p.checks = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxChecks, p.M / (2 * max_groups(p))));
  const dim3 down((unsigned)((p.M + p.checks - 1) / p.checks), (unsigned)((p.rank + kUnitRank - 1) / kUnitRank),
                  (unsigned)p.slices);
  const cudaError_t e =
      p.checks == 1
          ? launch(f16 ? few_down_kernel<__half, true> : few_down_kernel<__nv_bfloat16, true>, down, p, stream)
          : launch(f16 ? few_down_kernel<__half, false> : few_down_kernel<__nv_bfloat16, false>, down, p, stream);
  if (e != cudaSuccess) return e;
  // As many shares of the columns as are resident at once, of a warp's 32 columns at least.
  const int64_t groups = max_groups(p), resident = (int64_t)up_ctas_per_sm(rank_class(p.rank)) * sms;
  const int64_t shares =
      std::max<int64_t>(1, std::min<int64_t>((p.N + 32 * kWarps - 1) / (32 * kWarps), resident / groups));
  const cudaError_t up = launch(f16 ? up_kernel<__half>(p.rank, elem_out) : up_kernel<__nv_bfloat16>(p.rank, elem_out),
                                dim3((unsigned)shares, (unsigned)groups, 1), p, stream);
  // (few_up leaves the counters at zero: without it, what few_down counted is cleared here)
  if (up != cudaSuccess) cudaMemsetAsync(p.counts, 0, 2 * sizeof(uint32_t), stream);
  return up;
}

}  // namespace gb300

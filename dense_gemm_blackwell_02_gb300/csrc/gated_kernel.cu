// The gated feed-forward block and its gradients:
//     G = X Wg^T,  U = X Wu^T,  H = act(G) * U                       (element by element)
//     dG = dH U act'(G),  dU = dH act(G)
//     dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
// X: M x K, Wg and Wu: N x K, H: M x N.  Sums in binary32 (Tensor Memory), rounded once to the
// outputs' type; dG and dU are rounded to the element type between the two steps of the backward
// pass, because the matrix instructions take 16-bit operands: half a step of each term, which over a
// long sum adds about as much error as the rounding of the result itself, and more where its terms
// cancel.  In fp16 their range is widened by scales of rows and columns (GatedRange).
//
// Many rows: a CTA pair computes a 256 x 256 accumulator (cta_group::2).  In the forward pass its
// columns are 128 of G and the same 128 of U: the leader loads rows of Wg, its peer rows of Wu, so
// that the two meet in one thread's registers and neither goes through memory.  The backward
// products read their operands as they lie: where the sum runs along the rows of a matrix its TMA
// boxes hold 64 columns x 64 rows and the descriptors say MN-major, so nothing is transposed.
// Bound by the tensor cores: forwards 8192 x 28672 x 8192 bf16 4560 us, 1690 TFLOP/s with the power
// limit reached; backwards 8192 x 14336 x 4096 bf16 2250 us alone (1710 TFLOP/s), 2500 for seconds
// on end.  256 x 28672 x 8192 fp16 streams 0.94 GB of weights in 160 to 182 us, 5.3 to 6.0 TB/s.
#include <algorithm>

#include "elements.cuh"
#include "gated_ptx.cuh"
#include "gemm_kernel.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "umma.cuh"
#include "wait.cuh"

namespace gb300 {

namespace {

// ---------------------------------------------------------------------- activation --
// The logistic function of x and of -x, both to the last bits also where they are tiny.
struct Logistic {
  float at, opposite;
};
__device__ __forceinline__ Logistic logistic(float x) {
  const float e = __expf(-fabsf(x));
  const float big = __fdividef(1.0f, 1.0f + e), small = e * big;
  return x < 0.0f ? Logistic{small, big} : Logistic{big, small};
}

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

template <int ACT>
__device__ __forceinline__ float gate_of(float g) {
  if constexpr (ACT == kGateSilu) return g * logistic(g).at;
  // g times the normal distribution, from its own side's tail
  else if constexpr (ACT == kGateGelu) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  // (1 + tanh y) / 2 is the logistic function of 2 y
  else if constexpr (ACT == kGateGeluTanh)
    return g * logistic(kTanhScale * g * fmaf(kTanhCube * g, g, 1.0f)).at;
  else return g < 0.0f ? 0.0f : g;  // (NaN stays NaN)
}

// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ float2 gate_and_slope(float g) {
  if constexpr (ACT == kGateSilu) {
    const Logistic s = logistic(g);
    return make_float2(g * s.at, s.at * fmaf(g, s.opposite, 1.0f));
  } else if constexpr (ACT == kGateGelu) {
    const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
    return make_float2(g * cdf, fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), cdf));
  } else if constexpr (ACT == kGateGeluTanh) {
    const Logistic s = logistic(kTanhScale * g * fmaf(kTanhCube * g, g, 1.0f));
    // (beyond 100 one side of the logistic function is 0: the slope is the other side then, and not
    // 0 times an infinity)
    const float near = fminf(fmaxf(g, -100.0f), 100.0f);
    return make_float2(g * s.at, s.at * fmaf(kTanhScale * near * s.opposite,
                                             fmaf(3.0f * kTanhCube, near * near, 1.0f), 1.0f));
  } else {
    return make_float2(g < 0.0f ? 0.0f : g, g > 0.0f ? 1.0f : 0.0f);
  }
}

// f(std::integral_constant<int, ACT>) for a kind known at run time.
template <typename F>
__device__ __forceinline__ void by_kind(int kind, F f) {
  switch (kind) {
    case kGateSilu: f(std::integral_constant<int, kGateSilu>{}); break;
    case kGateGelu: f(std::integral_constant<int, kGateGelu>{}); break;
    case kGateGeluTanh: f(std::integral_constant<int, kGateGeluTanh>{}); break;
    default: f(std::integral_constant<int, kGateRelu>{}); break;
  }
}

template <typename T>
constexpr int out_kind_of() {
  return std::is_same<T, __half>::value ? kOutF16 : kOutBF16;
}

// ---------------------------------------------------------------------- many rows --
struct PairLayout {
  static constexpr uint32_t kStages = 6;
  static constexpr uint32_t kEpiWarps = 8;
  static constexpr uint32_t kThreads = 32 * (2 + kEpiWarps);
  static constexpr uint32_t kOperand = 128 * 128;  // one operand's share of a stage, per CTA
  static constexpr uint32_t kBlock = 64 * 128;     // 64 columns x 64 rows of an MN-major operand
  static constexpr uint32_t kTx = 2 * 2 * kOperand;
  static constexpr uint32_t kBOff = kStages * kOperand;
  static constexpr uint32_t kCOff = 2 * kStages * kOperand;
  static constexpr uint32_t kStaging = 32 * 128;
  static constexpr uint32_t kBarOff = kCOff + kEpiWarps * kStaging;
  static constexpr uint32_t kClcSlots = 4;
  static constexpr uint32_t kNumBars = 2 * kStages + 5 + 2 * kClcSlots;
  static constexpr uint32_t kTmemSlotOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kAbortOff = kTmemSlotOff + 4;
  static constexpr uint32_t kClcOff = (kAbortOff + 4 + 15) & ~15u;
  static constexpr uint32_t kDynamicBytes = kClcOff + kClcSlots * 16 + 1024;
  static_assert(kDynamicBytes <= 227 * 1024, "shared memory over the per-block limit");
};

// Tile u of a launch: of which product (0: H or dX; 1, 2: dWg, dWu), its place, and the K blocks
// that it sums over: a slice of them where tiles are cut.
struct GatedTile {
  int32_t which, m_blk, n_blk, k_blocks, slice, kb0, kb1;
  __device__ __forceinline__ GatedTile(int32_t u, const GatedParams& p, bool back) {
    const int32_t own = p.product[0].tiles * p.slices;
    const int32_t v = p.first == 0 ? u - own : u;  // beyond, or of, the weights'
    const bool weights = p.first == 0 ? v >= 0 : u < 2 * p.product[1].tiles;
    const GatedProduct& d = p.product[weights ? 1 : 0];
    int32_t t = weights ? v : p.first == 0 ? u : u - 2 * p.product[1].tiles;
    which = 0;
    if (weights) {
      which = 1 + t / d.tiles;
      t -= (which - 1) * d.tiles;
    }
    k_blocks = d.k_blocks;
    slice = 0;
    kb0 = 0, kb1 = k_blocks;
    if (!weights) {
      if (back) kb1 *= 2;
      if (p.slices > 1) {
        slice = t / d.tiles;
        t -= slice * d.tiles;
        const int32_t all = kb1;
        kb0 = (int32_t)((int64_t)slice * all / p.slices);
        kb1 = (int32_t)((int64_t)(slice + 1) * all / p.slices);
      }
    }
    // groups of group_m tiles along M, walked along N: tiles that run together share rows of
    // both operands in L2
    const int32_t group = p.group_m * d.num_n, g = t / group;
    const int32_t first = g * p.group_m, gm = min(d.num_m - first, p.group_m);
    const int32_t r = t - g * group;
    m_blk = first + r % gm;
    n_blk = r / gm;
  }
};

// The forward pass hands its tiles out round robin.  Backwards dX's and the weights' are one launch,
// the longer ones first, and a pair that is done takes a tile whose CTAs have not started (cluster
// launch control, as grouped launches of the GEMM do): tiles of two lengths in two launches left
// pairs idle at both ends (1025 x 1401 x 2008 41 us).
template <typename T, bool BACK>
__global__ void __launch_bounds__(PairLayout::kThreads, 1)
    gated_pair_kernel(const __grid_constant__ GatedMaps maps, const __grid_constant__ GatedParams p) {
  using L = PairLayout;
  constexpr int OUT = out_kind_of<T>();
  constexpr int32_t kTileCols = BACK ? 256 : 128;  // of an output
  constexpr bool kScaled = BACK && std::is_same<T, __half>::value;  // (GatedRange)

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA = base, sB = base + L::kBOff, sC = base + L::kCOff, bar0 = base + L::kBarOff;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (L::kStages + s); };
  auto acc_full_bar = [&](uint32_t i) { return bar0 + 8u * (2 * L::kStages + i); };
  auto acc_empty_bar = [&](uint32_t i) { return bar0 + 8u * (2 * L::kStages + 2 + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * L::kStages + 4);
  const uint32_t clc_full = drain_bar + 8u, clc_empty = clc_full + 8u * L::kClcSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlotOff);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + L::kAbortOff);
  const uint32_t warp = warp_id(), lane = lane_id();
  const WaitCtl ctl{p.wait_limit_ns, p.status, abort_flag};
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int32_t stride = (int32_t)(gridDim.x / 2);
  const ClcLink clc{base + L::kClcOff, clc_full, clc_empty, 0};
  // A role's way through the tiles.
  struct Walk {
    int32_t u;
    uint32_t taken;
  };
  auto next = [&](Walk& w) {
    if (w.taken == 0) {
      w.u = (int32_t)(blockIdx.x / 2);
    } else if constexpr (BACK) {
      if (!clc_next<2>(clc, w.taken - 1, ctl, w.u)) return false;
    } else {
      w.u += stride;
    }
    ++w.taken;
    return w.u < p.units;
  };

  if (warp == 0 && lane == 0) {
    for (uint32_t s = 0; s < L::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(acc_full_bar(i), 1);
      mbar_init(acc_empty_bar(i), 2 * L::kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    for (uint32_t i = 0; i < L::kClcSlots; ++i) {
      mbar_init(clc_full + 8u * i, 1);
      mbar_init(clc_empty + 8u * i, 2 * (2 + L::kEpiWarps) - 1);  // both CTAs' roles, one MMA issuer
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    if (!BACK || p.product[0].tiles > 0) {
      tma_prefetch_desc(&maps.a[0]);
      tma_prefetch_desc(&maps.b[BACK ? 0 : rank]);
    } else {
      tma_prefetch_desc(&maps.across[0]);
      tma_prefetch_desc(&maps.x);
    }
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_addr(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer --
    uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0, asked = 0;
    bool ok = true;
    // A stage, once it is free: issue(A's place, B's place, barrier).
    auto fill = [&](auto issue) {
      if (!warp_wait_inl(empty_bar(stage), phase ^ 1u, ctl, kSiteEmpty)) return false;
      if (leader) mbar_arrive_expect_tx_elect(full_bar(stage), L::kTx);
      issue(sA + stage * L::kOperand, sB + stage * L::kOperand, mapa_shared(full_bar(stage), 0));
      armed |= 1u << stage;
      armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == L::kStages) stage = 0, phase ^= 1u;
      return true;
    };
    Walk w{0, 0};
    if constexpr (BACK) {
      while (ok && next(w)) {
        const GatedTile t(w.u, p, BACK);
        const int32_t a0 = t.m_blk * 256 + (int32_t)rank * 128, b0 = t.n_blk * 256 + (int32_t)rank * 128;
        if (t.which == 0) {
          for (int32_t i = t.kb0; ok && i < t.kb1; ++i) {
            const int32_t pass = i < t.k_blocks ? 0 : 1, k0 = (i - pass * t.k_blocks) * kBlockK;
            ok = fill([&](uint32_t a, uint32_t b, uint32_t bar) {
              tma_load_2d_pair_elect(b, &maps.b[pass], b0, k0, bar);
              tma_load_2d_pair_elect(b + L::kBlock, &maps.b[pass], b0 + 64, k0, bar);
              tma_load_2d_pair_elect(a, &maps.a[pass], k0, a0, bar);
            });
          }
        } else {
          const CUtensorMap* mapA = &maps.across[t.which - 1];
          if constexpr (kScaled)
            if (__ldcg(p.range.copied + t.m_blk)) mapA = &maps.scaled[t.which - 1];
          for (int32_t i = 0; ok && i < t.k_blocks; ++i)
            ok = fill([&](uint32_t a, uint32_t b, uint32_t bar) {
              tma_load_2d_pair_elect(b, &maps.x, b0, i * kBlockK, bar);
              tma_load_2d_pair_elect(b + L::kBlock, &maps.x, b0 + 64, i * kBlockK, bar);
              tma_load_2d_pair_elect(a, mapA, a0, i * kBlockK, bar);
              tma_load_2d_pair_elect(a + L::kBlock, mapA, a0 + 64, i * kBlockK, bar);
            });
        }
        if (ok) ok = clc_request<2>(clc, asked, leader, ctl);
        if (ok) ++asked;
      }
    } else {
      // One row of tiles: every weight is read by one tile, X by all.  Built twice, as in the GEMM.
      auto produce = [&](auto hinted) {
        constexpr bool kHint = decltype(hinted)::value;
        const uint64_t pol_a = kHint ? l2_policy_evict_last() : 0ull, pol_b = kHint ? l2_policy_evict_first() : 0ull;
        while (ok && next(w)) {
          const GatedTile t(w.u, p, BACK);
          const int32_t a0 = t.m_blk * 256 + (int32_t)rank * 128, b0 = t.n_blk * 128;
          for (int32_t i = t.kb0; ok && i < t.kb1; ++i)
            ok = fill([&](uint32_t a, uint32_t b, uint32_t bar) {
              if constexpr (kHint) {
                tma_load_2d_pair_hint_elect(b, &maps.b[rank], i * kBlockK, b0, bar, pol_b);
                tma_load_2d_pair_hint_elect(a, &maps.a[0], i * kBlockK, a0, bar, pol_a);
              } else {
                tma_load_2d_pair_elect(b, &maps.b[rank], i * kBlockK, b0, bar);
                tma_load_2d_pair_elect(a, &maps.a[0], i * kBlockK, a0, bar);
              }
            });
        }
      };
      if (p.product[0].num_m == 1) produce(std::true_type{});
      else produce(std::false_type{});
    }
    // no copy may still be landing in shared memory when the CTA exits (the peer's complete on
    // the leader's barriers; after an abort they are given time)
    if (lane == 0) {
      if (leader) {
        for (uint32_t s = 0; s < L::kStages; ++s)
          if (armed & (1u << s)) wait_parity_drain(full_bar(s), (armed_phase >> s) & 1u, ctl);
        // nor an answer (after an abort one may be under way)
        if (asked > 0) wait_parity_drain(clc_full + 8u * ((asked - 1u) & 3u), ((asked - 1u) >> 2) & 1u, ctl);
      } else if (*abort_flag) {
        pause_ns(200000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer --
    if (leader) {
      constexpr uint32_t kIdesc = idesc_f16_kmajor(256, 256, std::is_same<T, __nv_bfloat16>::value);
      const uint64_t along_a = smem_desc_sw128_kmajor(sA), along_b = smem_desc_sw128_kmajor(sB);
      const uint64_t across_a = smem_desc_sw128_mnmajor(sA, L::kBlock), across_b = smem_desc_sw128_mnmajor(sB, L::kBlock);
      uint32_t stage = 0, phase = 0, iter = 0;
      bool ok = !p.test_stall || warp_wait(drain_bar, 0, ctl, kSiteTestStall);
      Walk w{0, 0};
      while (ok && next(w)) {
        const GatedTile t(w.u, p, BACK);
        const uint32_t slot = iter & 1u, d = tmem + slot * 256;
        if (!warp_wait_inl(acc_empty_bar(slot), ((iter >> 1) & 1u) ^ 1u, ctl, kSiteAccEmpty)) break;
        tc_fence_after();
        // `issue` of (the stage's place in descriptors, whether to add, its empty barrier)
        auto multiply = [&](int32_t k_blocks, auto issue) {
          for (int32_t kb = 0; kb < k_blocks; ++kb) {
            if (!warp_wait_inl(full_bar(stage), phase, ctl, kSiteFull)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue((uint64_t)((stage * L::kOperand) >> 4), kb > 0 ? 1u : 0u, empty_bar(stage));
            if (++stage == L::kStages) stage = 0, phase ^= 1u;
          }
        };
        if constexpr (!BACK) {
          multiply(t.kb1 - t.kb0, [&](uint64_t at, uint32_t add, uint32_t bar) {
            umma_stage_steps_elect<2, 2, 2>(d, along_a + at, along_b + at, kIdesc, add, bar);
          });
        } else if (t.which == 0) {
          multiply(t.kb1 - t.kb0, [&](uint64_t at, uint32_t add, uint32_t bar) {
            umma_stage_steps_elect<2, 2, 128>(d, along_a + at, across_b + at, kIdesc | kIdescBMnMajor, add, bar);
          });
        } else {
          multiply(t.k_blocks, [&](uint64_t at, uint32_t add, uint32_t bar) {
            umma_stage_steps_elect<2, 128, 128>(d, across_a + at, across_b + at,
                                                kIdesc | kIdescAMnMajor | kIdescBMnMajor, add, bar);
          });
        }
        if (ok) umma_commit_pair_elect(acc_full_bar(slot), 0x3);
        ++iter;
      }
      // every MMA issued must finish before Tensor Memory is released
      umma_commit_elect<2>(drain_bar);
      if (lane == 0) wait_parity_drain(drain_bar, 0, ctl);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue --
    const uint32_t q = warp & 3u, h = (warp - 2) >> 2;  // lane quarter, column half
    const uint32_t staging = sC + (warp - 2) * L::kStaging;
    uint32_t iter = 0;
    // 64 columns of the warp's 32 rows, from column n0 of output `o` on
    auto emit = [&](const float (&v)[64], int o, int32_t m0, int32_t n0) {
      const int32_t M = p.product[BACK && o > 0 ? 1 : 0].M, N = p.product[BACK && o > 0 ? 1 : 0].N;
      if (p.tma_store) {
        if (lane == 0) bulk_wait_group_read<0>();  // the box's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(staging + lane * 128u + ((c ^ (lane & 7u)) << 4),
                       pack2<OUT>(v[8 * c], v[8 * c + 1]), pack2<OUT>(v[8 * c + 2], v[8 * c + 3]),
                       pack2<OUT>(v[8 * c + 4], v[8 * c + 5]), pack2<OUT>(v[8 * c + 6], v[8 * c + 7]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && n0 < N && m0 < M) {
          tma_store_2d(&maps.out[o], staging, n0, m0);
          bulk_commit_group();
        }
      } else {
        store_piece_rows<OUT>(p.out[o], M, N, m0, n0, v, staging);
        store_piece_rows<OUT>(p.out[o], M, N, m0, n0 + 32, v + 32, staging);
      }
    };
    // The same of slice `s` of a cut tile (part 0 or, forwards, U's 1), unrounded.
    auto leave = [&](const float (&v)[64], int32_t s, int part, int32_t m0, int32_t n0) {
      const int32_t m = m0 + (int32_t)lane;
      const int64_t rows = (int64_t)(BACK ? s : 2 * s + part) * p.product[0].M + m;
      float* to = p.partial + rows * p.partial_pitch + n0;
#pragma unroll
      for (int c = 0; c < 64; c += 4)
        if (m < p.product[0].M && n0 + c < p.partial_pitch)
          *reinterpret_cast<float4*>(to + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
      __syncwarp();
    };
    // 64 columns of the accumulator
    auto fetch = [&](uint32_t at, float (&v)[64]) {
      uint32_t a[32], b[32];
      tmem_ld_32x32b_x32(at, a);
      tmem_ld_32x32b_x32(at + 32, b);
      tmem_ld_wait(a);
      tie_regs(b);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(a[j]), v[32 + j] = __uint_as_float(b[j]);
    };
    Walk w{0, 0};
    for (; next(w); ++iter) {
      const GatedTile t(w.u, p, BACK);
      const uint32_t slot = iter & 1u;
      const int32_t m0 = t.m_blk * 256 + (int32_t)(rank * 128 + q * 32);
      [[maybe_unused]] float back = 1.0f;  // what takes the scale of this lane's row back, asked for early
      if constexpr (kScaled) {
        const int32_t m = m0 + (int32_t)lane, rows = p.product[t.which == 0 ? 0 : 1].M;
        if (m < rows) {
          const int64_t i = t.which == 0 ? m : p.range.first_column + (int64_t)(t.which - 1) * rows + m;
          back = __ldcg(p.range.back + i);
          if (h == 0 && t.n_blk == 0 && t.slice == 0) p.range.most[i] = 0;  // (the next call's)
        }
      }
      if (!warp_wait_inl(acc_full_bar(slot), (iter >> 1) & 1u, ctl, kSiteAccFull)) break;
      tc_fence_after();
      const uint32_t at = tmem + ((q * 32u) << 16) + slot * 256;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(acc_empty_bar(slot), 0));
      };
      float v[64];
      if constexpr (!BACK) {
        const int32_t n0 = t.n_blk * kTileCols + (int32_t)h * 64;
        fetch(at + h * 64, v);
        if (p.slices > 1) {
          leave(v, t.slice, 0, m0, n0);
          fetch(at + 128 + h * 64, v);
          release();
          leave(v, t.slice, 1, m0, n0);
          continue;
        }
        by_kind(p.act, [&](auto kind) {
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = gate_of<decltype(kind)::value>(v[j]);
        });
        {
          float up[64];
          fetch(at + 128 + h * 64, up);
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] *= up[j];
        }
        if (p.outs == 1) release();
        emit(v, 0, m0, n0);
        if (p.outs > 1) {  // the projections too, as the gradients need them
          fetch(at + h * 64, v);
          emit(v, 1, m0, n0);
          fetch(at + 128 + h * 64, v);
          release();
          emit(v, 2, m0, n0);
        }
      } else {
        const int32_t n0 = t.n_blk * kTileCols + (int32_t)h * 128;
        const bool cut = p.slices > 1 && t.which == 0;
        auto scale_back = [&] {
          if constexpr (kScaled) {
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] *= back;
          }
        };
        fetch(at + h * 128, v);
        scale_back();
        if (cut) leave(v, t.slice, 0, m0, n0);
        else emit(v, t.which, m0, n0);
        fetch(at + h * 128 + 64, v);
        release();
        scale_back();
        if (cut) leave(v, t.slice, 0, m0, n0 + 64);
        else emit(v, t.which, m0, n0 + 64);
      }
    }
    // every TMA store of this warp must be complete before the CTA exits
    if (p.tma_store && lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
}

// The slices of cut tiles added up in their order, four columns a thread: H (and G and U), or dX.
constexpr int kJoinThreads = 256;
template <typename T, bool BACK>
__global__ void __launch_bounds__(kJoinThreads) gated_join_kernel(const GatedParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int32_t M = p.product[0].M, N = p.product[0].N, quads = p.partial_pitch / 4;
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int64_t m = i / quads;
  if (m >= M) return;
  const int32_t n = (int32_t)(i - m * quads) * 4;
  const int64_t part = (int64_t)M * p.partial_pitch;
  const float* from = p.partial + m * p.partial_pitch + n;
  constexpr int kParts = BACK ? 1 : 2;
  float sum[kParts][4] = {};
#pragma unroll 4
  for (int32_t s = 0; s < p.slices; ++s)
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(from + (int64_t)(kParts * s + q) * part);
      sum[q][0] += v.x, sum[q][1] += v.y, sum[q][2] += v.z, sum[q][3] += v.w;
    }
  auto put = [&](void* out, const float (&v)[4]) {
    T* to = static_cast<T*>(out) + m * N + n;
    if (p.tma_store) {  // (rows start on 16 bytes)
      store_f32<T, 4>(to, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < N) to[j] = from_f32<T>(v[j]);
    }
  };
  if constexpr (BACK) {
    put(p.out[0], sum[0]);
  } else {
    float h[4];
    by_kind(p.act, [&](auto kind) {
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = gate_of<decltype(kind)::value>(sum[0][j]) * sum[1][j];
    });
    put(p.out[0], h);
    if (p.outs > 1) {
      put(p.out[1], sum[0]);
      put(p.out[2], sum[1]);
    }
  }
}

// ----------------------------------------------------------------------- few rows --
// Up to 128 rows of X are the MMA's columns, and 8 to 128 rows of each weight its rows: a CTA
// streams those once, past all of X.  G and U of one column then lie in the same lane of two
// accumulators.  The tiles are made as narrow as spreads them over the SMs evenly (N 28672: two
// rounds of 96 rows on 150 SMs), and X comes from L2.  An MMA costs the same however few rows of
// it are a tile's, so where N is small K is cut too (launch_gated_few): the slices of a tile are a
// cluster, leave their sums in shared memory, and each of them adds up its share of X's rows, in
// the slices' order.  Bound by HBM where the weights are large (1 x 14336 x 4096 bf16 37.5 us,
// 6.3 TB/s), else by the latency of one tile (77 x 1001 x 2008 fp16 8.2 us, 16 without slices).
constexpr uint32_t kFewThreads = 32 * 10;
constexpr uint32_t kFewMaxStages = 16;
constexpr uint32_t kFewSmem = 227 * 1024;

template <typename T>
__global__ void __launch_bounds__(kFewThreads, 1)
    gated_few_kernel(const __grid_constant__ GatedFewMaps maps, const __grid_constant__ GatedFewParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bar_mem[2 * kFewMaxStages + 5];
  __shared__ uint32_t tmem_mem;
  __shared__ int32_t abort_mem;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t stages = (uint32_t)p.stages;
  const uint32_t w_bytes = (uint32_t)p.tile_rows * 128u, x_bytes = (uint32_t)p.x_rows * 128u;
  // all stages' rows of Wg, then of Wu, then of X: an MMA reads 128 rows of a weight from where
  // its stage starts, and those past the tile's rows feed lanes that nobody reads
  const uint32_t sG = base, sU = sG + stages * w_bytes, sX = sU + stages * w_bytes;
  const uint32_t bar0 = smem_addr(bar_mem);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kFewMaxStages + s); };
  auto acc_full_bar = [&](uint32_t i) { return bar0 + 8u * (2 * kFewMaxStages + i); };
  auto acc_empty_bar = [&](uint32_t i) { return bar0 + 8u * (2 * kFewMaxStages + 2 + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kFewMaxStages + 4);
  const uint32_t warp = warp_id(), lane = lane_id();
  const WaitCtl ctl{p.wait_limit_ns, p.status, &abort_mem};
  // (one tile per cluster: one slot of accumulators, so that the next launch's CTA fits beside it)
  const uint32_t tmem_cols = p.splits > 1 ? 256u : 512u;
  const int32_t slice = p.splits > 1 ? (int32_t)cluster_ctarank() : 0;
  const int32_t first = (int32_t)blockIdx.x / p.splits, stride = (int32_t)gridDim.x / p.splits;
  const int32_t kb0 = (int32_t)((int64_t)slice * p.k_blocks / p.splits);
  const int32_t kb1 = (int32_t)((int64_t)(slice + 1) * p.k_blocks / p.splits);

  if (warp == 0 && lane == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(acc_full_bar(i), 1);
      mbar_init(acc_empty_bar(i), 8);
    }
    mbar_init(drain_bar, 1);
    abort_mem = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.gate);
    tma_prefetch_desc(&maps.up);
    tma_prefetch_desc(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_addr(&tmem_mem), tmem_cols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_mem;
  grid_dependency_wait();
  grid_launch_dependents();

  float* partial = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)));
  // one value of every output
  auto put = [&](auto kind, int32_t m, int32_t n, float g, float w) {
    const int64_t i = (int64_t)m * p.N + n;
    static_cast<T*>(p.h)[i] = from_f32<T>(gate_of<decltype(kind)::value>(g) * w);
    if (p.gate) {
      static_cast<T*>(p.gate)[i] = from_f32<T>(g);
      static_cast<T*>(p.up)[i] = from_f32<T>(w);
    }
  };
  if (warp == 0) {
    uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    // the weights are read once, X by every CTA
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    for (int32_t u = first; ok && u < p.tiles; u += stride) {
      for (int32_t kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_inl(empty_bar(stage), phase ^ 1u, ctl, kSiteEmpty)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx_elect(full_bar(stage), 2 * w_bytes + x_bytes);
        tma_load_2d_hint_elect(sG + stage * w_bytes, &maps.gate, kb * kBlockK, u * p.tile_rows,
                               full_bar(stage), pol_w);
        tma_load_2d_hint_elect(sU + stage * w_bytes, &maps.up, kb * kBlockK, u * p.tile_rows,
                               full_bar(stage), pol_w);
        tma_load_2d_hint_elect(sX + stage * x_bytes, &maps.x, kb * kBlockK, 0, full_bar(stage), pol_x);
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
    }
    if (lane == 0)
      for (uint32_t s = 0; s < stages; ++s)
        if (armed & (1u << s)) wait_parity_drain(full_bar(s), (armed_phase >> s) & 1u, ctl);
    __syncwarp();
  } else if (warp == 1) {
    const uint64_t desc_g = smem_desc_sw128_kmajor(sG), desc_u = smem_desc_sw128_kmajor(sU),
                   desc_x = smem_desc_sw128_kmajor(sX);
    uint32_t stage = 0, phase = 0, iter = 0;
    bool ok = !p.test_stall || warp_wait(drain_bar, 0, ctl, kSiteTestStall);
    for (int32_t u = first; ok && u < p.tiles; u += stride, ++iter) {
      const uint32_t slot = iter & 1u;
      if (!warp_wait_inl(acc_empty_bar(slot), ((iter >> 1) & 1u) ^ 1u, ctl, kSiteAccEmpty)) break;
      tc_fence_after();
      for (int32_t kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_inl(full_bar(stage), phase, ctl, kSiteFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        umma_stage_twice_elect(tmem + slot * 256, tmem + slot * 256 + 128,
                               desc_g + ((stage * w_bytes) >> 4), desc_u + ((stage * w_bytes) >> 4),
                               desc_x + ((stage * x_bytes) >> 4), p.idesc, kb > kb0 ? 1u : 0u,
                               empty_bar(stage));
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      if (ok) umma_commit_elect<1>(acc_full_bar(slot));
    }
    umma_commit_elect<1>(drain_bar);
    if (lane == 0) wait_parity_drain(drain_bar, 0, ctl);
    __syncwarp();
  } else {
    const uint32_t q = warp & 3u, half = (warp - 2) >> 2;
    const int32_t row = (int32_t)(q * 32 + lane);
    uint32_t iter = 0;
    for (int32_t u = first; u < p.tiles; u += stride, ++iter) {
      const uint32_t slot = iter & 1u;
      if (!warp_wait_inl(acc_full_bar(slot), (iter >> 1) & 1u, ctl, kSiteAccFull)) break;
      tc_fence_after();
      const uint32_t at = tmem + ((q * 32u) << 16) + slot * 256;
      const int32_t n = u * p.tile_rows + row;
      const bool mine = row < p.tile_rows && n < p.N;
      if (q * 32 < (uint32_t)p.tile_rows) {
        // eight rows of X at a time, in turn by the quarter's two warps
        for (int32_t m0 = (int32_t)half * 8; m0 < p.M; m0 += 16) {
          uint32_t g[8], w[8];
          tmem_ld_32x32b_x8_async(at + (uint32_t)m0, g);
          tmem_ld_32x32b_x8_async(at + 128u + (uint32_t)m0, w);
          tmem_ld_wait(g, w);
          if (p.splits > 1) {  // (the ring is idle: all MMAs have read it)
            if (row < p.tile_rows) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                partial[(m0 + j) * p.tile_rows + row] = __uint_as_float(g[j]);
                partial[(p.x_rows + m0 + j) * p.tile_rows + row] = __uint_as_float(w[j]);
              }
            }
            continue;
          }
          by_kind(p.act, [&](auto kind) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (mine && m0 + j < p.M)
                put(kind, m0 + j, n, __uint_as_float(g[j]), __uint_as_float(w[j]));
          });
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty_bar(slot));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, tmem_cols);
  }
  if (p.splits > 1) {
    __syncwarp();
    cluster_sync();
    // this CTA's share of X's rows
    const int32_t m0 = (int32_t)((int64_t)slice * p.M / p.splits), m1 = (int32_t)((int64_t)(slice + 1) * p.M / p.splits);
    const uint32_t from = smem_addr(partial);
    by_kind(p.act, [&](auto kind) {
      for (int32_t i = (int32_t)threadIdx.x; i < (m1 - m0) * p.tile_rows; i += (int32_t)kFewThreads) {
        const int32_t m = m0 + i / p.tile_rows, row = i % p.tile_rows, n = first * p.tile_rows + row;
        float x[8], y[8], g = 0.0f, w = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          x[s] = y[s] = 0.0f;
          if (s >= p.splits) continue;
          const uint32_t at = mapa_shared(from + 4u * (uint32_t)(m * p.tile_rows + row), (uint32_t)s);
          x[s] = ld_cluster_f32(at);
          y[s] = ld_cluster_f32(at + 4u * (uint32_t)(p.x_rows * p.tile_rows));
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) g += x[s], w += y[s];
        if (n < p.N) put(kind, m, n, g, w);
      }
    });
    __syncwarp();
    cluster_sync();  // the others have read this CTA's sums
  }
}

// ------------------------------------------------------------------ the activation's gradient --
// Three reads and two writes per element, a handful of operations (some forty for Phi): bound by
// HBM where the arrays are large.  A thread takes
// eight results of a row.  Where rows start anywhere (VEC 0), their inputs are two aligned vectors
// apiece, moved together by the bytes between (1025 x 1401 fp16, kernel alone 11.5 us element by
// element).
constexpr int kSlopeThreads = 256;

// Eight elements from `at` on, of an array that ends at `end`.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, 8> eight_at(const T* at, const T* begin, const T* end) {
  if constexpr (VEC) {
    return *reinterpret_cast<const Pack<T, 8>*>(at);
  } else {
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(at) & 15u;
    const T* low = at - off / sizeof(T);
    Pack<T, 8> x;
    if (low >= begin && end - low >= 16) {
      const uint4 a = reinterpret_cast<const uint4*>(low)[0], b = reinterpret_cast<const uint4*>(low)[1];
      uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = off & 4u ? w[i + 1] : w[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2u) * 8u);
      *reinterpret_cast<uint4*>(&x) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x.v[j] = end - at > j ? at[j] : from_f32<T>(0.0f);
    }
    return x;
  }
}

// Row m's dG and dU from column n on, zeros behind the N-th.
template <typename T, int VEC>
__device__ __forceinline__ void slopes_at(const GatedSlopeParams& p, int64_t m, int32_t n, float (&dg)[8],
                                          float (&du)[8]) {
  const int64_t most = p.M * p.N, at = m * p.N + n;
  const T* dh_in = static_cast<const T*>(p.dh);
  const T* gate_in = static_cast<const T*>(p.gate);
  const T* up_in = static_cast<const T*>(p.up);
  float dh[8], g[8], up[8];
  unpack(eight_at<T, VEC>(dh_in + at, dh_in, dh_in + most), dh);
  unpack(eight_at<T, VEC>(gate_in + at, gate_in, gate_in + most), g);
  unpack(eight_at<T, VEC>(up_in + at, up_in, up_in + most), up);
  by_kind(p.act, [&](auto kind) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 a = gate_and_slope<decltype(kind)::value>(g[j]);
      dg[j] = VEC || n + j < p.N ? dh[j] * up[j] * a.y : 0.0f;
      du[j] = VEC || n + j < p.N ? dh[j] * a.x : 0.0f;
    }
  });
}

// f(row, column) of this thread's vectors.
template <typename F>
__device__ __forceinline__ void each_vector(const GatedSlopeParams& p, F f) {
  const uint32_t per_row = (uint32_t)p.pitch / 8;
  for (int64_t c = (int64_t)blockIdx.x * kSlopeThreads; c < p.M * per_row; c += (int64_t)gridDim.x * kSlopeThreads) {
    const int64_t m0 = c / per_row;  // (of the CTA's first vector)
    const uint32_t i = (uint32_t)(c - m0 * per_row) + threadIdx.x, down = i / per_row;
    const int64_t m = m0 + down;
    if (m >= p.M) break;
    f(m, (int32_t)(i - down * per_row) * 8);
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kSlopeThreads) gated_slope_kernel(const GatedSlopeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  each_vector(p, [&](int64_t m, int32_t n) {
    float dg[8], du[8];
    slopes_at<T, VEC>(p, m, n, dg, du);
    store_f32<T, 8>(static_cast<T*>(p.dgate) + m * p.pitch + n, dg);
    store_f32<T, 8>(static_cast<T*>(p.dup) + m * p.pitch + n, du);
  });
}

// fp16 (GatedRange): the same, unscaled, with the largest magnitudes of rows and columns.  A warp takes
// 256 columns of every eighth row of its CTA's: a row's largest is one reduction of the warp, a
// column's stays in a lane's registers; both meet the other CTAs' in memory, where the products leave
// zeros for the next call.  (An infinity may be the largest: what its row's or column's others are
// then scaled to does not matter, because the sums are infinite or NaN, and a NaN is none.)
// Measured, with the kernel behind it: 1025 x 1401 8.9 and 4.3 us each alone (the kernel above 6.2), the
// whole gradients 29 -> 34 us, 38.4 where rows and columns are scaled; 1024 x 4096 x 2048 50 -> 57 and
// 67; 8192 x 14336 x 4096 within the spread of 2300 to 2390, and 2720 to 2790.
constexpr int kRangeColumns = 256, kRangeWarps = kSlopeThreads / 32;

// 1 / scale of a row or column.
__device__ __forceinline__ float back_of(uint32_t most) {
  if (most == 0 || (most >= __float_as_uint(0x1p-4f) && most < __float_as_uint(0x1p15f))) return 1.0f;
  return __uint_as_float((max(most >> 23, 27u) - 14u) << 23);
}
__device__ __forceinline__ float scale_of(float back) {  // (a power of two's inverse)
  return __uint_as_float((254u << 23) - __float_as_uint(back));
}

// A CTA's and a lane's place in both kernels.
struct RangePlace {
  int32_t block, stripe, n0, n;
  int64_t first;  // the warp's first row
  __device__ __forceinline__ explicit RangePlace(const GatedSlopeParams& p) {
    const uint32_t stripes = (uint32_t)(p.pitch + kRangeColumns - 1) / kRangeColumns;
    block = (int32_t)(blockIdx.x / stripes);
    stripe = (int32_t)(blockIdx.x - (uint32_t)block * stripes);
    n0 = stripe * kRangeColumns;
    n = n0 + ((int)threadIdx.x & 31) * 8;
    first = (int64_t)block * kRangeWarps * p.row_steps + ((int)threadIdx.x >> 5);
  }
};

template <int VEC>
__global__ void __launch_bounds__(kSlopeThreads, 4) gated_slope_range_kernel(const GatedSlopeParams p) {
  __shared__ alignas(16) float columns[kRangeWarps][2][kRangeColumns];
  grid_dependency_wait();
  grid_launch_dependents();
  const RangePlace at(p);
  const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t n = at.n;
  float of_g[8] = {}, of_u[8] = {};
#pragma unroll 2
  for (int32_t step = 0; step < p.row_steps; ++step) {
    const int64_t m = at.first + (int64_t)step * kRangeWarps;
    if (m >= p.M) break;
    float most = 0.0f;
    if (n < p.pitch) {
      float dg[8], du[8];
      slopes_at<__half, VEC>(p, m, n, dg, du);
      store_f32<__half, 8>(static_cast<__half*>(p.dgate) + m * p.pitch + n, dg);
      store_f32<__half, 8>(static_cast<__half*>(p.dup) + m * p.pitch + n, du);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        of_g[j] = fmaxf(of_g[j], fabsf(dg[j])), of_u[j] = fmaxf(of_u[j], fabsf(du[j]));
        most = fmaxf(most, fmaxf(fabsf(dg[j]), fabsf(du[j])));
      }
    }
    if (p.range.rows) {
      const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
      if (lane == 0 && bits > 0) atomicMax(p.range.most + m, bits);
    }
  }
  if (p.range.columns) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(&columns[warp][0][lane * 8 + j]) = make_float4(of_g[j], of_g[j + 1], of_g[j + 2], of_g[j + 3]);
      *reinterpret_cast<float4*>(&columns[warp][1][lane * 8 + j]) = make_float4(of_u[j], of_u[j + 1], of_u[j + 2], of_u[j + 3]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float most = 0.0f;
#pragma unroll
      for (int w = 0; w < kRangeWarps; ++w) most = fmaxf(most, columns[w][k][tid]);
      const int32_t c = at.n0 + tid;
      if (most > 0.0f && c < p.N)
        atomicMax(p.range.most + p.range.first_column + (int64_t)k * p.N + c, __float_as_uint(most));
    }
  }
}

// ... the scales, and what has to be scaled, written, by CTAs of the same places: rows where their others
// are; a stripe's columns in their own copy, all of them once one of them or any row is scaled.  Mostly
// nothing has to be.
template <int VEC>
__global__ void __launch_bounds__(kSlopeThreads) gated_slope_scale_kernel(const GatedSlopeParams p) {
  __shared__ float scales[2][kRangeColumns];
  grid_dependency_wait();
  grid_launch_dependents();
  const RangePlace at(p);
  const GatedRange& r = p.range;
  const int tid = (int)threadIdx.x, lane = tid & 31;
  // this warp's rows, one for each lane
  const int64_t own = at.first + (int64_t)lane * kRangeWarps;
  float row = 1.0f;
  if (r.rows && lane < p.row_steps && own < p.M) {
    row = back_of(__ldcg(r.most + own));
    if (at.stripe == 0) r.back[own] = row;
  }
  bool copied = false;
  if (r.columns) {
    bool off = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int32_t c = at.n0 + tid;
      const int64_t i = r.first_column + (int64_t)k * p.N + c;
      const float back = c < p.N ? back_of(__ldcg(r.most + i)) : 1.0f;
      if (c < p.N && at.block == 0) r.back[i] = back;
      scales[k][tid] = scale_of(back);
      off |= back != 1.0f;
    }
    if (r.rows) {
#pragma unroll 4
      for (int32_t q = tid; q < r.first_column / 4; q += kSlopeThreads) {
        const uint4 most = __ldcg(reinterpret_cast<const uint4*>(r.most) + q);
        off |= back_of(most.x) != 1.0f || back_of(most.y) != 1.0f || back_of(most.z) != 1.0f || back_of(most.w) != 1.0f;
      }
    }
    copied = __syncthreads_or(off) != 0;
    if (at.block == 0 && tid == 0) r.copied[at.stripe] = copied;
  }
  if (copied || __any_sync(0xFFFFFFFFu, row != 1.0f)) {
    for (int32_t step = 0; step < p.row_steps; ++step) {
      const int64_t m = at.first + (int64_t)step * kRangeWarps;
      const float back = __shfl_sync(0xFFFFFFFFu, row, step);
      if (m >= p.M || at.n >= p.pitch || (!copied && back == 1.0f)) continue;
      float dg[8], du[8], g[8], u[8];
      slopes_at<__half, VEC>(p, m, at.n, dg, du);
      if (back != 1.0f) {
        const float s = scale_of(back);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = dg[j] * s, u[j] = du[j] * s;
        store_f32<__half, 8>(static_cast<__half*>(p.dgate) + m * p.pitch + at.n, g);
        store_f32<__half, 8>(static_cast<__half*>(p.dup) + m * p.pitch + at.n, u);
      }
      if (copied) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = dg[j] * scales[0][lane * 8 + j], u[j] = du[j] * scales[1][lane * 8 + j];
        store_f32<__half, 8>(static_cast<__half*>(p.dgate_by_column) + m * p.pitch + at.n, g);
        store_f32<__half, 8>(static_cast<__half*>(p.dup_by_column) + m * p.pitch + at.n, u);
      }
    }
  }
}

// --------------------------------------------------------- the weights' gradients of few rows --
// dWg and dWu are sums over M rows; for up to kGatedRankRows of them they are written as fast from
// binary32 operations as memory takes them, and dG and dU enter unrounded: with one row a rounding
// of dG would be that of a whole row of dWg.  A thread holds eight columns of X's rows; the CTA
// computes dG and dU of 64 columns at a time into shared memory, and every thread multiplies.
// Measured: 14336 x 4096 bf16 39 us with one row, 45 with eight (6.0 and 5.3 TB/s), in tiles 65.
// (Beside dX's kernel instead of before it: 130 us together with one row, 95 in turn.)
constexpr int kRankThreads = 256, kRankBatch = 64;

template <typename T, int R>
__global__ void __launch_bounds__(kRankThreads) gated_rank_kernel(const __grid_constant__ GatedRankParams p) {
  __shared__ float2 slopes[kRankBatch][R];  // dG and dU
  grid_dependency_wait();
  grid_launch_dependents();
  const int32_t i = (int32_t)threadIdx.x % p.cols, sub = (int32_t)threadIdx.x / p.cols, subs = kRankThreads / p.cols;
  const int64_t k = ((int64_t)blockIdx.x * p.cols + i) * 8;
  const bool mine = k < p.K;
  float x[R][8];
#pragma unroll
  for (int m = 0; m < R; ++m) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[m][j] = 0.0f;
    if (mine && m < p.M) unpack(*reinterpret_cast<const Pack<T, 8>*>(static_cast<const T*>(p.x) + m * p.K + k), x[m]);
  }
  const int64_t first = (int64_t)blockIdx.y * p.chunk, last = min(first + p.chunk, p.N);
  for (int64_t n0 = first; n0 < last; n0 += kRankBatch) {
    const int count = (int)min((int64_t)kRankBatch, last - n0);
    __syncthreads();  // the last batch has been read
    for (int e = (int)threadIdx.x; e < R * kRankBatch; e += kRankThreads) {
      const int m = e / kRankBatch, j = e % kRankBatch;
      float2 d = make_float2(0.0f, 0.0f);
      if (m < p.M && j < count) {
        const int64_t at = m * p.N + n0 + j;
        const float dh = to_f32(static_cast<const T*>(p.dh)[at]);
        const float g = to_f32(static_cast<const T*>(p.gate)[at]), up = to_f32(static_cast<const T*>(p.up)[at]);
        by_kind(p.act, [&](auto kind) {
          const float2 a = gate_and_slope<decltype(kind)::value>(g);
          d = make_float2(dh * up * a.y, dh * a.x);
        });
      }
      slopes[j][m] = d;
    }
    __syncthreads();
    if (!mine) continue;
    for (int j = sub; j < count; j += subs) {
      float wg[8], wu[8];
#pragma unroll
      for (int m = 0; m < R; ++m) {
        const float2 d = slopes[j][m];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          wg[q] = m == 0 ? d.x * x[0][q] : fmaf(d.x, x[m][q], wg[q]);
          wu[q] = m == 0 ? d.y * x[0][q] : fmaf(d.y, x[m][q], wu[q]);
        }
      }
      const int64_t at = (n0 + j) * p.K + k;
      store_f32<T, 8>(static_cast<T*>(p.d_gate_weight) + at, wg);
      store_f32<T, 8>(static_cast<T*>(p.d_up_weight) + at, wu);
    }
  }
}

// --------------------------------------------------------------------------- launches --
cudaLaunchConfig_t config_of(unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                             cudaLaunchAttribute (&attr)[2], unsigned cluster) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}

template <typename T, bool BACK>
cudaError_t launch_pair(const GatedMaps& maps, const GatedParams& p, int sms, cudaStream_t stream) {
  auto kernel = gated_pair_kernel<T, BACK>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)PairLayout::kDynamicBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const int32_t pairs = BACK ? p.units : std::min(p.units, std::max(sms / 2, 1));
  const cudaLaunchConfig_t cfg =
      config_of(2u * (unsigned)pairs, PairLayout::kThreads, PairLayout::kDynamicBytes, stream, attr, 2);
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

template <typename T, bool BACK>
cudaError_t launch_join(const GatedParams& p, cudaStream_t stream) {
  const int64_t threads = (int64_t)p.product[0].M * (p.partial_pitch / 4);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      config_of((unsigned)((threads + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, stream, attr, 1);
  return cudaLaunchKernelEx(&cfg, gated_join_kernel<T, BACK>, p);
}

template <typename T>
cudaError_t launch_few(const GatedFewMaps& maps, const GatedFewParams& p, uint32_t smem, cudaStream_t stream) {
  auto kernel = gated_few_kernel<T>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kFewSmem - 1024));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config_of((unsigned)p.ctas, kFewThreads, smem, stream, attr, (unsigned)p.splits);
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

template <typename T>
cudaError_t launch_rank(GatedRankParams& p, int sms, cudaStream_t stream) {
  const int64_t vectors = p.K / 8;
  p.cols = 8;  // a thread's column of vectors for each of as many threads as K has, up to all
  while (p.cols < kRankThreads && p.cols < vectors) p.cols *= 2;
  const int64_t across = (vectors + p.cols - 1) / p.cols;
  // as many CTAs as give every SM eight, in whole batches
  const int64_t down = std::max<int64_t>(1, std::min<int64_t>((8 * (int64_t)sms + across - 1) / across, 65535));
  const int64_t batches = (p.N + kRankBatch - 1) / kRankBatch;
  p.chunk = (batches + down - 1) / down * kRankBatch;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config_of((unsigned)across, kRankThreads, 0, stream, attr, 1);
  cfg.gridDim.y = (unsigned)((p.N + p.chunk - 1) / p.chunk);
  return p.M == 1   ? cudaLaunchKernelEx(&cfg, gated_rank_kernel<T, 1>, p)
         : p.M == 2 ? cudaLaunchKernelEx(&cfg, gated_rank_kernel<T, 2>, p)
         : p.M <= 4 ? cudaLaunchKernelEx(&cfg, gated_rank_kernel<T, 4>, p)
                    : cudaLaunchKernelEx(&cfg, gated_rank_kernel<T, 8>, p);
}

template <int VEC>
cudaError_t launch_slope(int elem, GatedSlopeParams& p, int sms, cudaStream_t stream) {
  const int64_t want = (p.M * (p.pitch / 8) + kSlopeThreads - 1) / kSlopeThreads;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config_of((unsigned)std::min<int64_t>(want, (int64_t)sms * 16), kSlopeThreads, 0, stream, attr, 1);
  if (elem == kElemBF16) return cudaLaunchKernelEx(&cfg, gated_slope_kernel<__nv_bfloat16, VEC>, p);
  // rows of a warp: as many as leave every SM four CTAs, 32 at most; of those behind it, which mostly do
  // next to nothing, two (1025 x 1401, alone, 7.2 us with eight, 4.9 with two)
  const int64_t stripes = (p.pitch + kRangeColumns - 1) / kRangeColumns, eights = (p.M + kRangeWarps - 1) / kRangeWarps;
  auto steps = [&](int64_t per_sm) {
    p.row_steps = (int32_t)std::max<int64_t>(1, std::min<int64_t>(32, eights * stripes / (per_sm * sms)));
    cfg.gridDim.x = (unsigned)((eights + p.row_steps - 1) / p.row_steps * stripes);
  };
  steps(4);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gated_slope_range_kernel<VEC>, p);
  if (e != cudaSuccess) return e;
  steps(2);
  return cudaLaunchKernelEx(&cfg, gated_slope_scale_kernel<VEC>, p);
}

}  // namespace

cudaError_t launch_gated(bool back, int elem, const GatedMaps& maps, const GatedParams& p, int sms,
                         cudaStream_t stream) {
  if (elem == kElemF16)
    return back ? launch_pair<__half, true>(maps, p, sms, stream) : launch_pair<__half, false>(maps, p, sms, stream);
  return back ? launch_pair<__nv_bfloat16, true>(maps, p, sms, stream)
              : launch_pair<__nv_bfloat16, false>(maps, p, sms, stream);
}

cudaError_t launch_gated_join(bool back, int elem, const GatedParams& p, cudaStream_t stream) {
  if (elem == kElemF16) return back ? launch_join<__half, true>(p, stream) : launch_join<__half, false>(p, stream);
  return back ? launch_join<__nv_bfloat16, true>(p, stream) : launch_join<__nv_bfloat16, false>(p, stream);
}

// In K blocks of a pair (a quarter of a microsecond): the end of the longest tile, or the average
// if that is later, without and with slices, against the join's 22 and what its sums' way through
// memory costs, 1.3 per megabyte; another tile's epilogue counts 10.  Both sides in us, uncut first:
// forwards 200 x 2048 x 7168 38.8 and 27.8, 256 x 4096 x 14336 69.6 and 55.3, 600 x 1024 x 4096
// 26.2 and 24.6, but 200 x 4096 x 2048 19.5 and 23.6, 129 x 4096 x 4096 26.7 and 28.1; gradients of
// 64 x 2048 x 2048 26.6 and 21.5, but of 300 x 4096 x 4096 51.2 and 61.4.
int32_t gated_slices(const GatedProduct& d, int64_t blocks, int64_t sums, int64_t others, int sms) {
  const int64_t pairs = std::max(sms / 2, 1);
  if (d.tiles == 0 || d.tiles >= pairs) return 1;
  const int64_t average = (d.tiles * blocks + others + pairs - 1) / pairs;
  const int64_t slices = std::min(std::min(pairs / d.tiles, blocks / 8), std::min<int64_t>(16, (blocks + average - 1) / average));
  if (slices < 2) return 1;
  const double bytes = 4.0 * (double)(slices * sums) * (double)d.M * (double)d.N;
  const int64_t gain = blocks - std::max((blocks + slices - 1) / slices, average);
  return (double)gain > 22.0 + 1.3e-6 * bytes ? (int32_t)slices : 1;
}

cudaError_t launch_gated_few(int elem, const GatedFewMaps& maps, GatedFewParams p, cudaStream_t stream) {
  // As many stages as shared memory holds.  The MMAs of the last stage of Wu read 128 rows from
  // its start, past the tile's rows and into X's, which hold them.
  const uint32_t stage = (uint32_t)(2 * p.tile_rows + p.x_rows) * 128u;
  // Short K slices leave room for the next launch's CTAs, which then set up before this one ends
  // (77 x 1001 x 2008 13.1 -> 8.2 us); longer ones want the stages (128 x 4096 x 4096 27 us with
  // half of them, 22.5 with all).
  const uint32_t half = kFewSmem / 2 - 4096, whole = kFewSmem - 4096;  // without alignment, static memory
  const bool compact = p.splits > 1 && (uint32_t)((p.k_blocks + p.splits - 1) / p.splits) <= 2 * (half / stage);
  p.stages = (int32_t)std::min(kFewMaxStages, (compact ? half : whole) / stage);
  p.stages = std::max(1, std::min(p.stages, (p.k_blocks + p.splits - 1) / p.splits));
  const uint32_t ring = (uint32_t)p.stages * stage;
  const uint32_t reach = (uint32_t)(2 * p.stages - 1) * (uint32_t)p.tile_rows * 128u + 128u * 128u;
  const uint32_t sums = p.splits > 1 ? (uint32_t)(2 * p.x_rows * p.tile_rows) * 4u : 0u;
  // Above half of an SM's memory, so that no two of these CTAs share one, each of which takes all of
  // Tensor Memory; with slices, which take half of it, above a third, so that no three do, nor one
  // beside a kernel that takes all: a cluster whose CTAs waited for Tensor Memory on one SM and held
  // it on another could wait for one that does the reverse, on another stream, for ever.
  const uint32_t smem = std::max(std::max(ring, sums), std::max(reach, compact ? kFewSmem / 3 : kFewSmem / 2)) + 1024u;
  return elem == kElemF16 ? launch_few<__half>(maps, p, smem, stream)
                          : launch_few<__nv_bfloat16>(maps, p, smem, stream);
}

GatedFewSplit gated_few_split(int64_t M, int64_t N, int64_t K, int sms) {
  // Rounds of tiles on the SMs, whole K: as few rows per tile as make the rounds even.
  const int64_t x_rows = (M + 15) / 16 * 16, k_blocks = (K + kBlockK - 1) / kBlockK;
  const int64_t rounds = (N + 128 * (int64_t)sms - 1) / (128 * (int64_t)sms);
  auto rows_of = [&](int64_t tiles) { return std::min<int64_t>(128, ((N + tiles - 1) / tiles + 7) / 8 * 8); };
  GatedFewSplit best{(int32_t)rows_of(rounds * sms), 1};
  // In microseconds at 1.9 GHz: a K block's eight MMAs take x_rows / 2 cycles each, its operands
  // come at about 50 bytes per cycle and SM, the weights at 6.5 TB/s; joining slices costs 2 us.  Fitted to
  // rank the choices, not to predict their times (128 x 4096 x 4096 comes to 12 us, measured 22.5).
  const double stream = 4e-6 * (double)N * (double)K / 6.5;
  auto cost = [&](int64_t rows, int64_t splits, int64_t times) {
    const double blocks = (double)((k_blocks + splits - 1) / splits * times);
    const double mma = blocks * 4.0 * (double)x_rows, ingest = blocks * (double)(2 * rows + x_rows) * 128.0 / 50.0;
    return std::max(std::max(mma, ingest) / 1900.0, stream) + (splits > 1 ? 2.0 : 0.0);
  };
  double least = cost(best.tile_rows, 1, rounds);
  // (clusters of 4 and 8 CTAs leave some SMs of each processing cluster without one)
  const int64_t clusters[3] = {sms / 2, sms * 36 / 152, sms * 16 / 152};
  for (int i = 0; i < 3; ++i) {
    const int64_t splits = 2ll << i;
    if (clusters[i] < 1 || N > 128 * clusters[i] || k_blocks < 2 * splits) continue;
    const int64_t rows = rows_of(clusters[i]);
    const double c = cost(rows, splits, 1);
    if (c < least) least = c, best = {(int32_t)rows, (int32_t)splits};
  }
  return best;
}

cudaError_t launch_gated_rank(int elem, GatedRankParams p, int sms, cudaStream_t stream) {
  return elem == kElemF16 ? launch_rank<__half>(p, sms, stream) : launch_rank<__nv_bfloat16>(p, sms, stream);
}

cudaError_t launch_gated_slope(int elem, GatedSlopeParams p, int sms, cudaStream_t stream) {
  return p.vec ? launch_slope<1>(elem, p, sms, stream) : launch_slope<0>(elem, p, sms, stream);
}

}  // namespace gb300

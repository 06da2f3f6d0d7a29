// Kernel parameter block and device status codes shared by the kernels and the
// host dispatcher (internal; the public interface is include/gemm.h).
#pragma once
#include <cuda.h>

#include <cstdint>

namespace gb300 {

// Tile edge along K of one pipeline stage: 64 x 16-bit = 128 bytes, the row of the
// 128-byte swizzle atom ("A Blackwell GEMM by Hand in CuTe DSL", section 6).
constexpr int kBlockK = 64;
// Rows of C per CTA (the M of a cta_group::1 MMA; half of a pair's 256).
constexpr int kBlockM = 128;
// Longest run of k-blocks accumulated in one TMEM accumulator before the epilogue
// folds it into its fp32 registers (64 x 64 = K 4096).  The tensor core's fp32
// accumulation error grows linearly with the length of one accumulation chain
// (measured: relative Frobenius error 4.0e-6 at K = 4096, 1.8e-5 at 16384, 3.2e-5
// at 28672 for U[-1,1] inputs); capping the chain keeps it near the K = 4096 value.
constexpr int kChainKBlocks = 64;

enum OutKind : int { kOutF16 = 0, kOutBF16 = 1, kOutF32 = 2 };

// Device status word: 0 = fine; otherwise (code << 24) | (site << 16) | blockIdx.x.
enum DeviceCode : uint32_t {
  kDevTimeout = 1u,   // a wait ran out (site: WaitSite)
  kDevBadIndex = 2u,  // an index in device memory was out of range (site: IndexSite)
};
enum IndexSite : uint32_t {
  kSiteRowAdapter = 1,  // row_adapter[i] >= count
  kSitePosition = 2,    // a rotary position outside the tables
  kSiteMaskRow = 3,     // mask_row[i] >= mask_count
};
enum WaitSite : uint32_t {
  kSiteEmpty = 1,     // producer waiting for a free stage
  kSiteFull = 2,      // MMA issuer waiting for a loaded stage
  kSiteAccEmpty = 3,  // MMA issuer waiting for a drained accumulator slot
  kSiteAccFull = 4,   // epilogue waiting for a finished accumulator
  kSiteTestStall = 5, // deliberate wait on a barrier nothing arrives on (test only)
  kSiteDrain = 6,     // teardown: outstanding copies / MMAs
  kSiteKx = 7,        // two-slice exchange through distributed shared memory
  kSiteClc = 8,       // cluster launch control: a free answer slot, or the next answer
  kSiteAdapterFull = 9,   // adapters: MMA issuer waiting for a loaded stage
  kSiteAdapterEmpty = 10, // adapters: producer waiting for a free stage
  kSiteAdapterAcc = 11,   // adapters: epilogue waiting for the finished accumulator
};

// One problem of a grouped launch ("CUTLASS Deep Dive: From CuTe Layouts to Blackwell
// tcgen05", Part 6, Grouped GEMM: each tile fetches its problem's pointers and tensor
// maps).  Written by the host into device memory; aligned as its tensor maps require.
struct GroupDesc {
  CUtensorMap tmA;        // A_g: box {128 bytes of K, 128 (or M_g < 128) rows}
  CUtensorMap tmB;        // B_g: box {128 bytes of K, BN / CTA_GROUP rows}
  CUtensorMap tmC;        // C_g: box {128 bytes of columns, 32 rows} (when tma_store)
  void* C;
  int32_t M, N, K;
  int32_t k_blocks;       // ceil(K_g / K block)
  int32_t num_m, num_n;   // tiles of this problem along M and N
  uint32_t a_tx_short;    // as GemmParams::a_tx_short, for this problem
  int32_t vec_store;      // 16-byte vector stores of C_g are aligned
  int32_t tma_store;      // C_g is written through tmC
};

// Adapters inside a product (the ADAPT kernels): the adapters that the rows of a 256-row
// tile name, and for each the rows that do not name it.
struct AdapterSlot {
  int32_t adapter;
  int32_t pad[3];
  uint32_t disable[8];    // bit r % 32 of word r / 32: row r of the tile does not name it
};
struct AdapterTile {
  int32_t slots;
  int32_t pad[3];
  AdapterSlot slot[2 * kBlockM];
};

// The 16-bit parts whose sum is u, the binary32 intermediate of an adapter, in the second
// product's operand type.  Each is the nearest to what the ones before leave: after two fp16
// parts at most 2^-23 of u is left, after two bf16 parts 2^-17, far below the rounding of a
// 16-bit result, and after three bf16 parts, for binary32 results, nothing.  (Parts of one sign,
// none of them zero, would keep infinities in Up as they are; but the matrix instructions'
// sums truncate, and such parts made even sums of small integers inexact.)
__host__ __device__ constexpr int u_parts(bool bf16_in, bool f32_out) {
  return bf16_in && f32_out ? 3 : 2;
}

constexpr int kAdaptCtas = 8;  // CTAs that share 128 rows in the kernel before, at most

// What an ADAPT kernel takes beside GemmParams; nothing in the others.
template <bool ADAPT>
struct AdaptParams {};
template <>
struct AdaptParams<true> {
  CUtensorMap tmU;        // u of every row, M x (64 * parts * ceil(rank / 64)), and as much again
                          // for the second window where there can be one: box {64, 128}
  CUtensorMap tmUp;       // (adapters * N) x rank: box {64, BN / 2}
  CUtensorMap tmUpHalf;   // ... box {64, BN / 4} (half-tile units)
  const AdapterTile* tiles;
  const float* row_scale; // M: of each row's term (RowFactor), 0 without an adapter
  const float* row_scale_low;  // M: of its second window
  const uint32_t* low;    // kAdaptCtas per 128 rows: whether one of the rows that a CTA of the
                          // kernel before saw to has a second window; nullptr: none can
  int32_t low_tiles, low_ctas;
  const float* u;         // M x rank
  const void* up;
  const int32_t* row_adapter;
  int32_t rank;
  int32_t parts;          // of u (u_parts)
  int32_t bf16;           // Up's type: bf16 or fp16
};

struct GemmParams {
  void* C;                 // M x N row-major output
  int32_t M, N, K;
  int32_t num_m_tiles;     // ceil(M / rows per tile); a tile is 128 * CTA_GROUP rows
  int32_t num_n_tiles;     // ceil(N / BN)
  int32_t tiles;           // num_m_tiles * num_n_tiles
  int32_t k_blocks;        // ceil(K / 64)
  int32_t dp_tiles;        // tiles [0, dp_tiles) run whole, one unit each
  int32_t half_tail;       // 1: each later tile runs as two BN/2-column halves (full K)
  int32_t splits;          // otherwise: K slices of each later tile (1 = no split)
  int32_t kb_per_split;    // k-blocks per slice (the last slice may be shorter)
  int32_t units;           // dp_tiles + (tiles - dp_tiles) * (half_tail ? 2 : splits)
  int32_t sk_workers;      // > 0: tiles after dp_tiles go to stream-K over this many units
  int32_t ws_slots;        // partial-tile slots per cut tile in the workspace
  int32_t group_m;         // grouped rasterisation: M-tiles per group
  int32_t chain_kb;        // k-blocks per TMEM accumulation chain
  int32_t prefetch_kb;     // L2 prefetch of B this many k-blocks ahead of the ring (0: off)
  int32_t l2_hint;         // 2: B's loads evict-first and A's evict-last in L2; else none
  uint32_t a_tx_short;     // bytes of A's 128-row box that A's tensor map does not load:
                           // (128 - M) * 128 when a one-CTA tile's A box is M < 128 rows
                           // (for the pair in the swapped tiling: 2 * (128 - swap_rows) * 128)
  int32_t swap_rows;       // swapped tiling (B is the MMA's row operand): B rows per CTA
  int32_t vec_store;       // 1 when 16-byte vector stores of C are aligned
  int32_t tma_store;       // 1 when C is written through the C tensor map
  uint32_t idesc;          // tcgen05 instruction descriptor (N = BN)
  uint32_t idesc_half;     // the same for N = BN / 2 (half-tile units)
  float* workspace;        // splits > 1: fp32 partial tiles
  uint32_t* counters;      // splits > 1: per (tile, CTA of the pair, quarter, half) counters
  uint32_t* status;        // device status word
  // fused epilogue, fused = 0: C = A . B^T; else C = act(alpha * A . B^T + beta * C + bias)
  int32_t fused;
  int32_t relu;            // act: ReLU when 1, the identity when 0
  float alpha, beta;
  const float* bias;       // N values (16-byte aligned), or nullptr
  // blockwise FP8 scales (KIND 2), K-block-major: sfa[kb * sf_lda + m / sf_bm],
  // sfb[kb * sf_ldb + n / 128]
  const float* sfa;
  const float* sfb;
  int32_t sf_bm, sf_lda, sf_ldb;
  // grouped launches (GROUPED kernels): problem g owns units [group_start[g],
  // group_start[g + 1]); units = group_start[num_groups]
  const GroupDesc* groups;
  const int32_t* group_start;
  int32_t num_groups;
  uint64_t wait_limit_ns;  // bound on every mbarrier wait
  int32_t test_stall;      // 1: the MMA issuer waits on a barrier that never completes
};

}  // namespace gb300

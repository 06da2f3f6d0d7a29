// Internal launch interface between operators_api.cu and the kernels of the operators
// around the projections: adapters, rotary positions, adjusted logits.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "params.h"

namespace gb300 {

// Element types, numbered as gemm_dtype_t's first three (which OutKind also follows).
enum ElemKind : int { kElemF16 = 0, kElemBF16 = 1, kElemF32 = 2 };

// ---------------------------------------------------------------------------- rotary --
constexpr int kMaxPairs = 256;  // rot_dim / 2

struct RotaryParams {
  const void* x;
  void* y;
  int64_t x_token, x_head, y_token, y_head;  // strides in elements
  int32_t tokens, heads, dim, half;          // half: pairs per head
  int32_t inverse;
  int32_t tile_tokens;  // tokens per CTA
  int32_t shares;       // CTAs per tile of tokens,
  int32_t share_heads;  // each this many heads
  int32_t items;        // work items per head: vectors of pairs, then vectors to copy
  const float* cos;
  const float* sin;
  const int32_t* positions;
  int64_t num_positions;
  uint32_t* status;
  alignas(8) uint8_t pair_axis[kMaxPairs];
};

// vec: 16-byte accesses of x, y and the tables are aligned and no vector straddles the
// pairs' end.  The split into CTAs is filled in here.
cudaError_t launch_rotary(RotaryParams p, int elem, bool neighbours, bool vec, int sms,
                          cudaStream_t stream);
int rotary_vector(int elem);  // elements of a 16-byte vector

// ---------------------------------------------------------------------------- logits --
struct LogitsParams {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;
  int32_t rows;
  int32_t vocab;
  int32_t slice;    // vocabulary entries per CTA (a multiple of 64)
  int32_t slices;   // CTAs per row
  const int32_t* tokens;
  const int64_t* token_start;
  const int32_t* prompt_len;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_tokens;
  const float* bias_values;
  const int64_t* bias_start;
  const uint32_t* mask;
  int64_t mask_stride, mask_count;
  const int32_t* mask_row;
  uint32_t* status;
};

// The split into CTAs is filled in here.
cudaError_t launch_logits(LogitsParams p, int elem_in, int elem_out, int sms, cudaStream_t stream);

// -------------------------------------------------------------------------- adapters --
constexpr int kMaxRank = 128;
constexpr int kAdapterRows = 128;   // rows of X per tile
constexpr int kAdapterCols = 128;   // columns of Down . X per group of adapters

// A batch of few rows (adapters_few_kernel.cu), queued right after the shared product.
constexpr int kFewRows = 512;
constexpr int kFewRowsLargePool = 2048;  // of a pool of more than kLargePool adapters
constexpr int kLargePool = 32;
constexpr int kFewGroup = 16;  // rows of one adapter that are taken together
struct FewGroup {
  int32_t adapter;          // -1: none
  int32_t rows;             // how many
  int32_t row[kFewGroup];   // -1 past them
  int32_t pad[14];          // 128 bytes
};
struct AdapterFewParams {
  const void* X;        // M x K, M <= kFewRowsLargePool
  const void* down;     // count x rank x K
  const void* up;       // count x N x rank
  const float* scale;   // count, or nullptr
  const int32_t* row_adapter;
  int32_t M, N, K, rank, count;
  int64_t base_pitch;   // values per row of base
  int32_t slices;       // partial sums of u (few_slices)
  int32_t checks;       // rows that a CTA of the first kernel looks at (set by the launch)
  int32_t vec_store;    // 16-byte accesses of eight columns of Y are aligned
  int32_t vec_base;     // rows of base start on 16 bytes
  float* partial;       // M x slices x rank
  FewGroup* groups;     // M
  uint32_t* counts;     // groups listed, CTAs that have read that; zero between calls
  const float* base;    // M x N: W . x; may be Y
  void* Y;              // M x N
  uint32_t* status;
};
int few_slices(int32_t M, int32_t K, int32_t rank, int32_t count, int sms);
// Rows of Down that the first kernel streams, at most.
int64_t few_down_rows(int32_t M, int32_t rank, int32_t count);
cudaError_t launch_adapter_few(AdapterFewParams p, int elem_in, int elem_out, int sms,
                               cudaStream_t stream);

// Many rows (adapters_kernel.cu): u of every row and the tiles' adapters, for the GEMM.
struct AdapterParams {
  const float* scale;   // count, or nullptr
  const int32_t* row_adapter;
  int32_t M, N, K, rank, count;
  int32_t tiles;        // ceil(M / kAdapterRows)
  int32_t k_blocks;     // ceil(K / 64)
  int32_t ctas;         // CTAs per row tile, a cluster: 1, 2, 4 or 8
  int32_t max_splits;   // K slices at most
  uint32_t idesc;       // instruction descriptor without N, 128 rows
  int32_t parts;        // of u (u_parts)
  int32_t f32_out;      // Y's type is binary32
  void* U;              // M x (64 * parts * ceil(rank / 64)) values of the input type, twice that
                        // in fp16, whose second half is the second window (RowFactor)
  float* row_scale;     // M (RowFactor)
  float* row_scale_low; // M
  uint32_t* low;        // kAdaptCtas per tile (AdaptParams)
  float* u;             // M x rank
  AdapterTile* pairs;   // ceil(tiles / 2)
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t test_stall;
};

// tmX: X, box {64, 128}; tmDown: (count * rank) x K, box {64, rank}.
cudaError_t launch_adapter_down(const CUtensorMap& tmX, const CUtensorMap& tmDown,
                                const AdapterParams& p, int elem_in, cudaStream_t stream);

// ------------------------------------------------------------- gated feed-forward --
enum GateKind : int { kGateSilu = 0, kGateGelu = 1, kGateGeluTanh = 2, kGateRelu = 3 };

// The products of the block, of CTA pairs with 256 x 256 accumulators (gated_kernel.cu).
// Forwards H (and the projections): X with 128 rows of Wg and of Wu, K along the rows of all.
// Backwards dX = dG Wg + dU Wu (K along the rows of dG and dU, across those of the weights) and
// dWg = dG^T X, dWu = dU^T X (K across the rows of both operands).
struct GatedMaps {
  CUtensorMap a[2];       // X; dG, dU: box {64, 128}
  CUtensorMap across[2];  // dG, dU: box {64, 64}
  CUtensorMap scaled[2];  // fp16: the same scaled by columns (GatedRange)
  CUtensorMap b[2];       // Wg, Wu: box {64, 128}, backwards {64, 64}
  CUtensorMap x;          // X: box {64, 64}
  CUtensorMap out[3];     // box {64, 32}
};
struct GatedProduct {
  int32_t M, N;           // rows and columns of the output
  int32_t num_m, num_n;   // tiles along them
  int32_t tiles;
  int32_t k_blocks;       // of one pair of operands
};
// fp16's range is too short for dG and dU (products of two values and a slope): a row of both, for dX,
// and a column of either, for the weights' gradients, whose largest lies outside
// 2^-4..2^15 is scaled by the power of two that brings it to 2^14..2^15, and its sums are scaled back.
// 2^-4 leaves a term an error of 2^-21 of that largest, if not of half its own step.
struct GatedRange {
  uint32_t* most;         // magnitudes' bit patterns: of M rows, from first_column on of dG's and of
                          // dU's N columns; zero between calls
  float* back;            // 1 / scale, laid out as `most`
  uint32_t* copied;       // of 256 columns each: in use is their scaled copy
  int64_t first_column;   // M rounded up to 4
  int32_t rows, columns;  // wanted (dX, the weights' gradients)
};

struct GatedParams {
  void* out[3];           // H, gate, up; dX, dWg, dWu: row-major, dense
  int32_t outs;           // forwards: how many of them
  GatedProduct product[2];  // forwards one; backwards dX, and either weight's (0 tiles: not wanted)
  int32_t first;          // backwards: whose tiles come first, 0 or 1
  int32_t slices;         // that the K blocks of H's or dX's tiles are cut into
  int32_t partial_pitch;  // with more than one: their sums' row pitch, a multiple of 4,
  float* partial;         // and the sums: slices (forwards of G and U in turn), M, pitch
  int32_t units;          // tiles of all products
  int32_t group_m;        // grouped rasterisation: tiles along M per group
  int32_t act;            // GateKind
  int32_t tma_store;      // the outputs are written through their maps
  GatedRange range;       // backwards in fp16
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t test_stall;
};
cudaError_t launch_gated(bool back, int elem, const GatedMaps& maps, const GatedParams& p, int sms,
                         cudaStream_t stream);
// Into how many slices the tiles of a product are cut that sum over `blocks` K blocks each, beside
// other tiles worth `others` blocks in all; the slices' sums (`sums` of them per value) are joined
// by a launch of its own.
int32_t gated_slices(const GatedProduct& d, int64_t blocks, int64_t sums, int64_t others, int sms);
cudaError_t launch_gated_join(bool back, int elem, const GatedParams& p, cudaStream_t stream);

// Few rows of X: weights streamed past them.
constexpr int kGatedFewRows = 128;
struct GatedFewMaps {
  CUtensorMap gate, up;  // Wg, Wu: box {64, tile_rows}
  CUtensorMap x;         // X: box {64, x_rows}
};
struct GatedFewParams {
  void* h;
  void* gate;            // the projections, or nullptr
  void* up;
  int32_t M, N;
  int32_t tile_rows;     // rows of each weight per tile, a multiple of 8, at most 128
  int32_t x_rows;        // M rounded up to 16
  int32_t tiles;
  int32_t k_blocks;
  int32_t splits;        // K slices of a tile, a cluster's CTAs: 1, 2, 4 or 8
  int32_t ctas;          // with slices splits for each tile
  int32_t stages;        // filled in by the launch
  int32_t act;
  uint32_t idesc;        // of 128 x x_rows
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t test_stall;
};
cudaError_t launch_gated_few(int elem, const GatedFewMaps& maps, GatedFewParams p, cudaStream_t stream);
// Rows of each weight per tile, and K slices.
struct GatedFewSplit {
  int32_t tile_rows, splits;
};
GatedFewSplit gated_few_split(int64_t M, int64_t N, int64_t K, int sms);

// dG = dH U act'(G) and dU = dH act(G), rounded to the element type: rows of `pitch` values, zeros
// behind the N-th.
struct GatedSlopeParams {
  const void* dh;
  const void* gate;
  const void* up;
  void* dgate;
  void* dup;
  int64_t M;
  int32_t N, pitch;
  int32_t act;
  int32_t vec;           // N is a multiple of 8 and the inputs start on 16 bytes
  // fp16
  GatedRange range;
  void* dgate_by_column; // where dG and dU scaled by columns go: dgate and dup if rows are not wanted
  void* dup_by_column;
  int32_t row_steps;     // filled in by the launch: rows of a warp
};
cudaError_t launch_gated_slope(int elem, GatedSlopeParams p, int sms, cudaStream_t stream);

// dWg and dWu of up to kGatedRankRows rows, dG and dU unrounded.
constexpr int32_t kGatedRankRows = 8;
struct GatedRankParams {
  const void* x;
  const void* dh;
  const void* gate;
  const void* up;
  void* d_gate_weight;
  void* d_up_weight;
  int64_t N, K;
  int32_t M;
  int32_t act;
  // filled in by the launch
  int32_t cols;          // threads along K
  int64_t chunk;         // rows of the weights per CTA
};
cudaError_t launch_gated_rank(int elem, GatedRankParams p, int sms, cudaStream_t stream);

// ------------------------------------------------------------------ normed and rotated heads --
constexpr int kMaxHeadDim = 512;
struct HeadsParams {
  const void* x;
  const void* dy;        // backwards
  void* y;               // backwards dx
  int64_t x_token, x_head, dy_token, dy_head, y_token, y_head;  // strides in elements
  int64_t tokens;
  int32_t heads, query_heads, dim, half;  // half: pairs per head
  const void* query_weight;  // dim values, or nullptr: all 1
  const void* key_weight;
  int32_t weight_elem;   // their type
  float eps, inv_dim;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  int64_t num_positions;
  float* partial;        // backwards: a row of dim sums for each CTA; nullptr: dw is not wanted
  float* d_query_weight;
  float* d_key_weight;
  uint32_t* status;
  // filled in by the launch
  int32_t items;         // of a head: vectors of pairs, then vectors of the rest
  int32_t lanes;         // of a head
  int32_t tile_tokens;   // tokens per CTA at a time
  int32_t key_tile_tokens;      // backwards, of the CTAs with key heads
  int32_t shares, share_heads;  // forwards: CTAs per tile, and their heads
  int32_t query_ctas, ctas;     // backwards
  alignas(8) uint8_t pair_axis[kMaxPairs];
};
int heads_back_ctas(int sms);  // rows of `partial` at most
// vec: elements per access (16 bytes' worth, 4, or 1) for which x, dy, y, the pairs and the rest
// of a head are aligned.
cudaError_t launch_heads(HeadsParams p, int elem, bool neighbours, int vec, int sms, cudaStream_t stream);
cudaError_t launch_heads_back(HeadsParams p, int elem, bool neighbours, int vec, int sms,
                              cudaStream_t stream);

// ------------------------------------------------------------------------ the next token --
struct SampleParams {
  const void* logits;
  int64_t stride;        // elements per row
  int32_t rows, vocab;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* random;
  int32_t* tokens;
  float* probs;          // or nullptr
  // filled in by the launch
  int32_t cluster;       // CTAs per row
  int32_t slice;         // logits per CTA
  int32_t resident;      // a slice stays in shared memory
  int32_t ahead;         // rows that run at once
  int32_t ordered;       // the rows that may take long run first
};
constexpr int32_t kMaxSampleVocab = 1 << 20;
cudaError_t launch_sample(SampleParams p, int elem, int sms, cudaStream_t stream);

}  // namespace gb300

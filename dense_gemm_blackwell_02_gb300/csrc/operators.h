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

}  // namespace gb300

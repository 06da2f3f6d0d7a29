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
  int32_t head_run;     // consecutive heads of one token that a thread turns
  int32_t head_runs;    // ceil(heads / head_run)
  int32_t items;        // work items per head: vectors of pairs, then vectors to copy
  const float* cos;
  const float* sin;
  const int32_t* positions;
  int64_t num_positions;
  uint32_t* status;
  alignas(8) uint8_t pair_axis[kMaxPairs];
};

// vec: 16-byte accesses of x, y and the tables are aligned and no vector straddles the
// pairs' end.  head_run, head_runs and items are filled in here.
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
  int32_t slice;    // vocabulary entries per CTA (a multiple of 32)
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

// slice and slices are filled in here.
cudaError_t launch_logits(LogitsParams p, int elem_in, int elem_out, int sms, cudaStream_t stream);

// -------------------------------------------------------------------------- adapters --
constexpr int kMaxRank = 128;

struct AdapterParams {
  const void* X;        // M x K
  const void* down;     // count x rank x K
  const void* up;       // count x N x rank
  const float* scale;   // count, or nullptr
  const int32_t* row_adapter;
  int32_t M, N, K, rank, count;
  float* U;             // M x rank: s * Down . x of every row with an adapter
  const float* base;    // M x N: W . x
  void* Y;              // M x N
  uint32_t* status;
};

cudaError_t launch_adapter_down(const AdapterParams& p, int elem_in, int sms, cudaStream_t stream);
cudaError_t launch_adapter_up(const AdapterParams& p, int elem_in, int elem_out, int sms,
                              cudaStream_t stream);

}  // namespace gb300

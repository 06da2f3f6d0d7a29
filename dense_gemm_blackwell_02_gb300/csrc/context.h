// The handle behind gemm_handle_t and the host helpers that the C ABI's translation units
// share (gemm_api.cu, operators_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <functional>

#include "gemm.h"
#include "params.h"
#include "scratch.h"

namespace gb300 {

constexpr int kTmapCacheSize = 16;

struct TmapKey {
  const void* ptr;
  int64_t rows, cols;
  int32_t dtype, box_rows;
  bool operator==(const TmapKey& o) const {
    return ptr == o.ptr && rows == o.rows && cols == o.cols && dtype == o.dtype &&
           box_rows == o.box_rows;
  }
};

struct TmapEntry {
  TmapKey key;
  CUtensorMap map;
  bool valid;
};

}  // namespace gb300

struct gemm_ctx {
  int device = 0;
  cudaError_t last_cuda = cudaSuccess;  // the CUDA error behind the last GEMM_ERR_CUDA launch
  int sms = 0;
  uint32_t* d_status = nullptr;
  gb300::Scratch ws;        // partial tiles of a product cut along K
  gb300::Scratch ctr;       // its arrival counters, zero between calls
  void* d_stage[3] = {nullptr, nullptr, nullptr};  // gemm_run_host: A, B, C
  size_t stage_bytes[3] = {0, 0, 0};
  gb300::Scratch op;        // scratch of the operators around the projections
  gb300::Scratch op_ctr;    // their counters, zero between calls
  gemm_config_t forced = {};
  int32_t short_chains = 0;  // K blocks per accumulation chain where none is forced (0: the default)
  // elements per row of C where not N: a whole number of 16 bytes; C is then written by TMA
  // alone (no swapped tiling, no 320-column tiles, nothing forced)
  int64_t c_pitch = 0;
  // rows of K values that another kernel streams beside the product (0: none does)
  int64_t beside_rows = 0;
  gemm_config_t last = {};
  uint64_t wait_limit_ns = 2000000000ull;
  int32_t test_stall = 0;
  gb300::TmapEntry cache[gb300::kTmapCacheSize] = {};
  int cache_next = 0;
  int resident[2][2][2][3] = {};  // [cta_group-1][bn==256][small A][out]: co-resident units (0: unknown)
  // gemm_plan: a device described instead of queried (resident CTA pairs, and clusters of
  // four CTAs for the pair's cluster K split); the GPU is never touched
  bool model = false;
  int model_pairs = 0, model_clusters4 = 0;
  // grouped launches: a ring of problem tables (pinned host copy, device copy and the
  // event that marks the host copy reusable)
  static constexpr int kGroupRing = 4;
  gb300::GroupDesc* h_groups[kGroupRing] = {};
  gb300::GroupDesc* d_groups[kGroupRing] = {};
  int32_t* h_gstart[kGroupRing] = {};
  int32_t* d_gstart[kGroupRing] = {};
  cudaEvent_t group_done[kGroupRing] = {};
  size_t group_cap[kGroupRing] = {};
  int group_next = 0;
  // gemm_run_host: copy streams and the events that order the chunks of the pipeline
  static constexpr int kHostChunks = 8;
  cudaStream_t copy_in = nullptr, copy_out = nullptr;
  cudaEvent_t host_ev[2 + 3 * kHostChunks] = {};
};

namespace gb300 {

// 2-D tensor map over a row-major rows x cols matrix, 128-byte swizzle, box of 128
// bytes of columns x box_rows rows.  Loads read out-of-range elements as zero (M, N and
// K tails); stores skip them.
bool make_map(gemm_ctx* h, const void* ptr, int64_t rows, int64_t cols, int dtype, int box_rows,
              CUtensorMap* out);

// The product of a CTA-pair kernel with low-rank adapters appended to its tiles.  `before`
// queues the kernel that prepares what `ad` points to, once the configuration is known to
// serve the shape.
gemm_status_t run_adapted(gemm_ctx* h, const void* A, const void* B, void* C, int64_t M, int64_t N,
                          int64_t K, gemm_dtype_t dtype_in, gemm_dtype_t dtype_out,
                          const AdaptParams<true>& ad, const std::function<cudaError_t()>& before,
                          gemm_stream_t stream);

}  // namespace gb300

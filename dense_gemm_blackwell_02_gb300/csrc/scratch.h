// Device memory that a handle owns and grows on demand.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>

#include "gemm.h"

namespace gb300 {

// Memory that is zero when the call returns, whichever stream uses it next.  (cudaMemset
// returns before the clearing is done, and streams that do not synchronise with the legacy
// one would not wait for it.)
inline gemm_status_t make_cleared(void** p, size_t bytes) {
  *p = nullptr;
  if (cudaMalloc(p, bytes) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OOM;
  }
  cudaStream_t s = nullptr;
  bool ok = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess;
  if (ok) {
    ok = cudaMemsetAsync(*p, 0, bytes, s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
    cudaStreamDestroy(s);
  }
  if (ok) return GEMM_OK;
  cudaGetLastError();
  cudaFree(*p);
  *p = nullptr;
  return GEMM_ERR_CUDA;
}

// A block that is replaced by a larger one when a call needs more.  The blocks it outgrew
// are kept until the handle goes: a captured graph still names them.  Each is at least twice
// the one before (unless memory is short), so all of them together are smaller than the last.
struct Scratch {
  static constexpr int kMaxOutgrown = 64;
  void* ptr = nullptr;
  size_t bytes = 0;
  struct {
    void* ptr;
    size_t bytes;
  } outgrown[kMaxOutgrown] = {};
  int num_outgrown = 0;

  // At least `want` bytes; zero in a new block if `cleared`.  On an error the old block stays.
  gemm_status_t grow(size_t want, bool cleared) {
    if (want <= bytes) return GEMM_OK;
    if (ptr && num_outgrown == kMaxOutgrown) return GEMM_ERR_OOM;
    gemm_status_t st = GEMM_ERR_OOM;
    void* p = nullptr;
    size_t size = 0;
    for (size_t n : {std::max(want, 2 * bytes), want}) {
      size = n;
      if (cleared) {
        st = make_cleared(&p, n);
      } else {
        st = cudaMalloc(&p, n) == cudaSuccess ? GEMM_OK : GEMM_ERR_OOM;
        if (st != GEMM_OK) cudaGetLastError();
      }
      if (st != GEMM_ERR_OOM) break;
    }
    if (st != GEMM_OK) return st;
    if (ptr) outgrown[num_outgrown++] = {ptr, bytes};
    ptr = p;
    bytes = size;
    return GEMM_OK;
  }
  // (asynchronous on the legacy stream)
  void clear() {
    for (int i = 0; i < num_outgrown; ++i) cudaMemset(outgrown[i].ptr, 0, outgrown[i].bytes);
    if (ptr) cudaMemset(ptr, 0, bytes);
  }
  void release() {
    for (int i = 0; i < num_outgrown; ++i) cudaFree(outgrown[i].ptr);
    if (ptr) cudaFree(ptr);
    *this = Scratch{};
  }
};

}  // namespace gb300

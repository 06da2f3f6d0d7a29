// Device memory that a handle owns and grows on demand.
#pragma once
#include <cuda_runtime.h>

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

}  // namespace gb300

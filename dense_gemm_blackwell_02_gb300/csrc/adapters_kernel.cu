// Low-rank adapters beside a shared projection, a different one for every row:
//     Y[i] = W . X[i] + s * Up[a] . (Down[a] . X[i]),   a = row_adapter[i]
// W . X comes from the GEMM in binary32 (`base`); the kernels here form
// u[i] = s * Down[a] . X[i] in binary32 and add Up[a] . u[i] to the base, rounding once.
#include <algorithm>

#include "elements.cuh"
#include "operators.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 256;

// The adapter of row i, or -1; an id past the pool is recorded and not followed.
__device__ __forceinline__ int32_t adapter_of(const AdapterParams& p, int32_t i) {
  const int32_t a = p.row_adapter[i];
  if (a < p.count) return a < 0 ? -1 : a;
  record_bad_index(p.status, kSiteRowAdapter);
  return -1;
}

// One CTA per row, one warp per value of u at a time: the lanes stride over K.
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_down_kernel(const AdapterParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int32_t i = (int32_t)blockIdx.x;
  const int32_t a = adapter_of(p, i);
  if (a < 0) return;
  const T* x = static_cast<const T*>(p.X) + (int64_t)i * p.K;
  const float s = p.scale ? p.scale[a] : 1.0f;
  for (int32_t r = (int32_t)warp_id(); r < p.rank; r += kThreads / 32) {
    const T* d = static_cast<const T*>(p.down) + ((int64_t)a * p.rank + r) * p.K;
    float acc = 0.0f;
    for (int32_t k = (int32_t)lane_id() * 8; k < p.K; k += 256) {
      float xv[8], dv[8];
      load_f32<T, 8>(x + k, xv);
      load_f32<T, 8>(d + k, dv);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = fmaf(xv[j], dv[j], acc);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, off);
    if (lane_id() == 0) p.U[(int64_t)i * p.rank + r] = s * acc;
  }
}

// One thread per element of Y.
template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads) adapter_up_kernel(const AdapterParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int32_t blocks = (p.N + kThreads - 1) / kThreads;
  const int32_t i = (int32_t)(blockIdx.x / (uint32_t)blocks);
  const int32_t n = (int32_t)(blockIdx.x - (uint32_t)i * (uint32_t)blocks) * kThreads + (int32_t)threadIdx.x;
  if (n >= p.N) return;
  const int32_t a = adapter_of(p, i);
  float acc = p.base[(int64_t)i * p.N + n];
  if (a >= 0) {
    const T* up = static_cast<const T*>(p.up) + ((int64_t)a * p.N + n) * p.rank;
    const float* u = p.U + (int64_t)i * p.rank;
    float d = 0.0f;
    for (int32_t r = 0; r < p.rank; r += 8) {
      float uv[8];
      load_f32<T, 8>(up + r, uv);
#pragma unroll
      for (int j = 0; j < 8; ++j) d = fmaf(u[r + j], uv[j], d);
    }
    acc += d;
  }
  static_cast<TO*>(p.Y)[(int64_t)i * p.N + n] = from_f32<TO>(acc);
}

template <typename K>
cudaError_t launch(K kernel, int64_t grid, const AdapterParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t up_by_out(const AdapterParams& p, int elem_out, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.M * ((p.N + kThreads - 1) / kThreads);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  switch (elem_out) {
    case kElemF16: return launch(adapter_up_kernel<T, __half>, grid, p, stream);
    case kElemBF16: return launch(adapter_up_kernel<T, __nv_bfloat16>, grid, p, stream);
    default: return launch(adapter_up_kernel<T, float>, grid, p, stream);
  }
}

}  // namespace

cudaError_t launch_adapter_down(const AdapterParams& p, int elem_in, int sms, cudaStream_t stream) {
  if (elem_in == kElemF16) return launch(adapter_down_kernel<__half>, p.M, p, stream);
  return launch(adapter_down_kernel<__nv_bfloat16>, p.M, p, stream);
}

cudaError_t launch_adapter_up(const AdapterParams& p, int elem_in, int elem_out, int sms,
                              cudaStream_t stream) {
  if (elem_in == kElemF16) return up_by_out<__half>(p, elem_out, stream);
  return up_by_out<__nv_bfloat16>(p, elem_out, stream);
}

}  // namespace gb300

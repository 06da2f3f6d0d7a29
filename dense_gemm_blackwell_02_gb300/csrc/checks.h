// Checks and small steps that the operators' entry points share (operators_api.cu,
// layer_api.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "context.h"
#include "gemm.h"

namespace gb300 {

inline bool valid_dtype(int d) { return d >= GEMM_F16 && d <= GEMM_E5M2; }
inline bool is_fp8(int d) { return d == GEMM_E4M3 || d == GEMM_E5M2; }
inline int64_t elem_size(int d) { return d == GEMM_F32 ? 4 : 2; }
inline bool aligned(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

// The handle's scratch for these operators, grown on demand; its counters are zero between
// calls.
inline gemm_status_t ensure_scratch(gemm_ctx* h, size_t bytes, size_t counters) {
  const gemm_status_t st = h->op.grow(bytes, false);
  return st != GEMM_OK ? st : h->op_ctr.grow(counters * sizeof(uint32_t), true);
}

// Whether two of n1 x n2 vectors of `dim` elements, s1 and s2 elements apart, share an element
// (n1 and n2 at least 1).
inline bool overlap(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t dim) {
  if (n1 == 1) std::swap(n1, n2), std::swap(s1, s2);  // (of a single one the stride does not count)
  if (n2 == 1) return n1 > 1 && s1 < dim;
  if (s1 > s2) std::swap(n1, n2), std::swap(s1, s2);
  if (s1 < dim) return true;
  // j steps of s2 against the nearest numbers of steps of s1, as far as those reach
  using wide = __int128;
  const wide reach = (wide)(n1 - 1) * s1 + dim;
  for (int64_t j = 1; j < n2 && (wide)j * s2 < reach; ++j) {
    const wide at = (wide)j * s2, past = at % s1;
    if (past < dim || (at / s1 + 1 < n1 && s1 - past < dim)) return true;
  }
  return false;
}

// Memory of n1 x n2 vectors of `bytes` each, s1 and s2 bytes apart (none negative).
struct Vectors {
  using wide = __int128;
  wide at, n1, s1, n2, s2, bytes;

  // The same memory with the larger stride first, without strides that lead nowhere and with vectors
  // that touch as one.
  Vectors joined() const {
    Vectors v = *this;
    if (v.s1 == 0) v.n1 = 1;
    if (v.s2 == 0) v.n2 = 1;
    if (v.n1 == 1) v.s1 = 0;
    if (v.n2 == 1) v.s2 = 0;
    if (v.s1 < v.s2) std::swap(v.n1, v.n2), std::swap(v.s1, v.s2);
    if (v.n2 > 1 && v.s2 <= v.bytes) v.bytes += (v.n2 - 1) * v.s2, v.n2 = 1, v.s2 = 0;
    if (v.n2 == 1 && v.n1 > 1 && v.s1 <= v.bytes) v.bytes += (v.n1 - 1) * v.s1, v.n1 = 1, v.s1 = 0;
    return v;
  }
  wide end() const { return at + (n1 - 1) * s1 + (n2 - 1) * s2 + bytes; }
  // Whether p..p + len - 1 meets any of them.
  bool meets(wide p, wide len) const {
    const wide from = p - at - bytes, to = p - at + len;  // a vector that begins between the two does
    if (to <= 0) return false;
    const wide reach = from - (n2 - 1) * s2;
    wide i = s1 == 0 || reach < 0 ? 0 : reach / s1 + 1;
    for (; i < n1 && i * s1 < to; ++i) {
      const wide rest = from - i * s1, j = rest < 0 ? 0 : s2 == 0 ? n2 : rest / s2 + 1;
      if (j < n2 && i * s1 + j * s2 < to) return true;
    }
    return false;
  }
};

// Whether a and b share a byte.
inline bool share_memory(const Vectors& a_, const Vectors& b_) {
  Vectors a = a_.joined(), b = b_.joined();
  if (a.at >= b.end() || b.at >= a.end()) return false;
  if (a.n1 == b.n1 && a.s1 == b.s1 && a.n2 == b.n2 && a.s2 == b.s2) {
    // (of one layout only the vectors' distances count: those of b from a's first, either way)
    b.at -= (a.n1 - 1) * a.s1 + (a.n2 - 1) * a.s2;
    b.n1 = 2 * a.n1 - 1, b.n2 = 2 * a.n2 - 1;
    return b.meets(a.at, a.bytes);
  }
  if (a.n1 * a.n2 > b.n1 * b.n2) std::swap(a, b);
  for (Vectors::wide i = 0; i < a.n1; ++i)
    for (Vectors::wide j = 0; j < a.n2; ++j)
      if (b.meets(a.at + i * a.s1 + j * a.s2, a.bytes)) return true;
  return false;
}

inline gemm_status_t launched(gemm_ctx* h, cudaError_t e) {
  h->last_cuda = e;
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

}  // namespace gb300

// A CUDA runtime that only keeps a journal, for tests of the library's host side on a
// machine without a GPU: the library's own object files are linked against it in place of
// the real runtime.  Device memory is host memory, kernels are recorded and not run, and
// the test reads the journal or makes a launch fail.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

namespace {

std::string journal;
std::map<const void*, std::string>& names() {  // (kernels register before this file's globals exist)
  static std::map<const void*, std::string>* m = new std::map<const void*, std::string>;
  return *m;
}
std::map<const void*, size_t> blocks;
std::string failing;  // part of the name of the kernel whose launches fail
size_t largest = ~(size_t)0;

void note(const char* what, const void* p, size_t n, const void* stream, const char* name = "") {
  char line[768];
  std::snprintf(line, sizeof(line), "%s %llx %zu %llx %.500s\n", what, (unsigned long long)(uintptr_t)p,
                n, (unsigned long long)(uintptr_t)stream, name);
  journal += line;
}

CUresult encode_nothing(CUtensorMap* m, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                        const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                        CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                        CUtensorMapFloatOOBfill) {
  std::memset(m, 0, sizeof(*m));
  return CUDA_SUCCESS;
}

}  // namespace

extern "C" {

// What the tests call.
const char* fake_journal() { return journal.c_str(); }
void fake_clear() { journal.clear(); }
void fake_fail(const char* part) { failing = part; }
void fake_largest(size_t n) { largest = n; }  // allocations above this fail

cudaError_t cudaMalloc(void** p, size_t n) {
  *p = nullptr;
  if (n > largest) return cudaErrorMemoryAllocation;
  *p = std::aligned_alloc(256, (n + 255) / 256 * 256);
  std::memset(*p, 0xA5, n);
  blocks[*p] = n;
  note("malloc", *p, n, nullptr);
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  if (p) note("free", p, blocks[p], nullptr);
  blocks.erase(p);
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned) {
  *p = std::malloc(n);
  return cudaSuccess;
}
cudaError_t cudaFreeHost(void* p) {
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int v, size_t n) {
  std::memset(p, v, n);
  note("memset", p, n, nullptr, "asynchronous on the legacy stream");
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) {
  if (blocks.count(p)) std::memset(p, v, n);
  note("memset", p, n, s);
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) {
  std::memcpy(d, s, n);
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() {
  note("synchronize-device", nullptr, 0, nullptr);
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) {
  note("synchronize", nullptr, 0, s);
  return cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned flags) {
  static uintptr_t next = 0x51000;
  *s = reinterpret_cast<cudaStream_t>(next += 0x10);
  note("stream", nullptr, flags, *s);
  return cudaSuccess;
}
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
  *e = reinterpret_cast<cudaEvent_t>(0xE000);
  return cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3
       : a == cudaDevAttrMultiProcessorCount ? 152 : 0;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "cudaErrorLaunchFailure"; }
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
  *p = nullptr;
  return cudaErrorInvalidValue;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&encode_nothing);
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = 1;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  const unsigned size = c->numAttrs ? c->attrs[c->numAttrs - 1].val.clusterDim.x : 1;
  *n = size >= 4 ? 36 : 76;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const std::string& name = names()[f];
  const bool fails = !failing.empty() && name.find(failing) != std::string::npos;
  note(fails ? "failed-launch" : "launch", nullptr, (size_t)c->gridDim.x * c->gridDim.y * c->gridDim.z,
       c->stream, name.c_str());
  return fails ? cudaErrorLaunchFailure : cudaSuccess;
}

// What the compiler's own code around the kernels calls.
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*,
                            dim3*, int*) {
  names()[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t __cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t __cudaGetKernel(void**, const void*) { return cudaSuccess; }

}  // extern "C"

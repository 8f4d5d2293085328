// A stand-in for the CUDA runtime under the library's own objects: no GPU, no
// kernel runs.  It keeps a log of what the host code asks for (in order, with
// the thread, the device and the stream), so that tests on the CPU can see what
// a GPU would be told: the order of launches, the memory they are given, the
// attributes of a kernel on each device.
#include <atomic>
#include <chrono>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>
#include <map>
#include <mutex>
#include <set>
#include <string>
#include <thread>
#include <vector>

namespace {
std::mutex mu;
std::string text;                                            // the log, a line an event
std::map<const void*, std::string> names;                    // kernels by their host stub
std::map<std::pair<int, const void*>, int> smem_allowed;     // by device
std::set<cudaStream_t> capturing;
std::map<void*, size_t> blocks;
std::atomic<int> launch_us{0};
std::atomic<int> next_thread{0};
thread_local int device = 0;
thread_local const int thread = next_thread++;

void log(const char* what, cudaStream_t st, const std::string& more) {
  char head[96];
  std::snprintf(head, sizeof head, "%s thread=%d device=%d stream=%llu ", what, thread, device,
                static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(st)));
  std::lock_guard<std::mutex> lock(mu);
  text += head + more + "\n";
}
std::string hex(const void* p) {
  char s[32];
  std::snprintf(s, sizeof s, "%llx", static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(p)));
  return s;
}
cudaError_t launch(const void* f, dim3 grid, size_t smem, cudaStream_t st) {
  std::string name;
  {
    std::lock_guard<std::mutex> lock(mu);
    name = names[f];
    // (what needs no opt-in on a GPU: 48 KB, a kernel's static part of up to 8 KB included)
    if (smem > 40 * 1024 && smem_allowed[{device, f}] < static_cast<int>(smem)) return cudaErrorInvalidValue;
  }
  if (const int us = launch_us) std::this_thread::sleep_for(std::chrono::microseconds(us));
  log("launch", st, name + " grid=" + std::to_string(grid.x));
  return cudaSuccess;
}
CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                     const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
// ---- what the tests set and read -------------------------------------------------
void fake_set_device(int d) { device = d; }
void fake_set_capturing(void* st, int on) {
  std::lock_guard<std::mutex> lock(mu);
  if (on) capturing.insert(static_cast<cudaStream_t>(st));
  else capturing.erase(static_cast<cudaStream_t>(st));
}
void fake_set_launch_us(int us) { launch_us = us; }
int fake_thread() { return thread; }
const char* fake_take_log() {
  static thread_local std::string out;
  std::lock_guard<std::mutex> lock(mu);
  out.swap(text);
  text.clear();
  return out.c_str();
}

// ---- the runtime -----------------------------------------------------------------
void** __cudaRegisterFatBinary(void*) {
  static void* handle = nullptr;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* stub, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) { names[stub] = name; }
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3, void**, size_t smem, cudaStream_t st) {
  return launch(reinterpret_cast<const void*>(k), grid, smem, st);
}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, cudaStream_t) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) { return launch(f, c->gridDim, c->dynamicSmemBytes, c->stream); }

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  std::lock_guard<std::mutex> lock(mu);
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) smem_allowed[{device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = 4;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = 8;
  return cudaSuccess;
}
cudaError_t cudaMallocAsync(void** p, size_t bytes, cudaStream_t st) {
  *p = std::calloc(1, bytes);
  if (!*p) return cudaErrorMemoryAllocation;
  {
    std::lock_guard<std::mutex> lock(mu);
    blocks[*p] = bytes;
  }
  log("malloc", st, hex(*p) + " bytes=" + std::to_string(bytes));
  return cudaSuccess;
}
cudaError_t cudaFreeAsync(void* p, cudaStream_t st) {
  log("free", st, hex(p));
  std::lock_guard<std::mutex> lock(mu);
  if (!blocks.erase(p)) return cudaErrorInvalidValue;
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t bytes, cudaStream_t st) {
  log("memset", st, hex(p) + " bytes=" + std::to_string(bytes));
  std::memset(p, v, bytes);
  return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int v, size_t bytes) {
  std::memset(p, v, bytes);
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* d, const void* s, size_t bytes, cudaMemcpyKind) {
  std::memcpy(d, s, bytes);
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t bytes, cudaMemcpyKind, cudaStream_t) {
  std::memcpy(d, s, bytes);
  return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t st, cudaStreamCaptureStatus* s) {
  std::lock_guard<std::mutex> lock(mu);
  *s = capturing.count(st) ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
// Not reached by what the tests call.
cudaError_t cudaEventCreate(cudaEvent_t*) { return cudaErrorNotSupported; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaErrorNotSupported; }
cudaError_t cudaEventElapsedTime(float*, cudaEvent_t, cudaEvent_t) { return cudaErrorNotSupported; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaErrorNotSupported; }
cudaError_t cudaMalloc(void**, size_t) { return cudaErrorNotSupported; }
cudaError_t cudaFree(void*) { return cudaErrorNotSupported; }
cudaError_t cudaGetSymbolAddress(void**, const void*) { return cudaErrorNotSupported; }
}

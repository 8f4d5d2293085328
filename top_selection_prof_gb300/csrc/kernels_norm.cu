// The norm of many tensors taken as one vector, and their scaling to a largest
// norm: n = sqrt(sum g^2), g <- g min(1, max_norm / (n + 1e-6)).
//
// The tensors are cut into chunks of kChunk values; the table of tensors goes
// to the kernel as its parameter, so nothing is copied to the device.  A block
// sums the squares of its chunks in f32 a thread at a time (at most
// kChunk / kThreads squares in one f32 sum), adds those in f64 and writes one
// partial sum; the last block adds all partial sums in their order.  Where the
// f32 squares of a chunk overflow, or are so small that bits are lost, the
// chunk is summed again in f64, so that the norm is exact to f32 for any
// finite input.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;        // values of a chunk
constexpr int kTable = 640;         // tensors of one launch (the kernel parameter holds their table)
constexpr int kMaxBlocks = 2048;

struct TensorTable {
  const void* in[kTable];
  void* out[kTable];
  int64_t count[kTable];
  uint32_t first[kTable + 1];  // first chunk of each tensor
  uint8_t f32[kTable];
  int tensors;
};
struct NormScratch {
  double* part;       // per block of this launch
  double* carry;      // sum of the launches before it
  unsigned* ticket;
  float* scale;
};

__device__ __forceinline__ int tensor_of(const TensorTable& t, uint32_t chunk) {
  int lo = 0, hi = t.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Calls f(value) for this thread's values of [p, p + n): whole 16-byte vectors
// between a head and a tail of single values.
template <typename T, typename F>
__device__ __forceinline__ void each_value(const T* p, int n, F f) {
  constexpr int kVec = 16 / sizeof(T);
  const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int(sizeof(T)));
  const int vecs = (n - head) / kVec;
  for (int i = threadIdx.x; i < head; i += kThreads) f(to_f32(p[i]));
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    Vec<T, kVec> v;
    v.load(p + head + i * kVec);
#pragma unroll
    for (int c = 0; c < kVec; ++c) f(v.v[c]);
  }
  for (int i = head + vecs * kVec + threadIdx.x; i < n; i += kThreads) f(to_f32(p[i]));
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
  float sum = 0.0f, most = 0.0f;
  each_value(p, n, [&](float v) {
    sum = fmaf(v, v, sum);
    most = fmaxf(most, fabsf(v));
  });
  // squares between 2^-100 and 2^126 / n lose nothing; NaN and inf stay what they are
  if (most == 0.0f || !(most < INFINITY) || (most > 1e-15f && most < 1e17f)) return static_cast<double>(sum);
  double wide = 0.0;
  each_value(p, n, [&](float v) { wide += static_cast<double>(v) * v; });
  return wide;
}

__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) t += shared[w];
  __syncthreads();
  return t;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ TensorTable t, NormScratch s,
                                                           bool first, bool finish, float max_norm, float* norm) {
  __shared__ double shared[kThreads / 32];
  __shared__ bool last;
  double sum = 0.0;
  const uint32_t chunks = t.first[t.tensors];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = int64_t(c - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(int64_t(kChunk), t.count[i] - at));
    sum += t.f32[i] ? chunk_squares(static_cast<const float*>(t.in[i]) + at, n)
                    : chunk_squares(static_cast<const __nv_bfloat16*>(t.in[i]) + at, n);
  }
  sum = block_sum(sum, shared);
  if (threadIdx.x == 0) {
    s.part[blockIdx.x] = sum;
    __threadfence();
    last = atomicAdd(s.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double all = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) all += __ldcg(&s.part[i]);
  all = block_sum(all, shared);
  if (threadIdx.x == 0) {
    if (!first) all += *s.carry;
    *s.carry = all;
    *s.ticket = 0;
    if (finish) {
      const float n = static_cast<float>(sqrt(all));
      *norm = n;
      const float f = max_norm / (n + 1e-6f);
      *s.scale = f > 1.0f ? 1.0f : f;  // (NaN stays NaN)
    }
  }
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* p, T* out, int n, float f) {
  constexpr int kVec = 16 / sizeof(T);
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) & 15, b = reinterpret_cast<uintptr_t>(out) & 15;
  const int head = a == b ? min(n, static_cast<int>((16 - a) & 15) / int(sizeof(T))) : n;
  const int vecs = (n - head) / kVec;
  for (int i = threadIdx.x; i < head; i += kThreads) out[i] = from_f32<T>(to_f32(p[i]) * f);
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    Vec<T, kVec> v;
    v.load(p + head + i * kVec);
#pragma unroll
    for (int c = 0; c < kVec; ++c) v.v[c] *= f;
    v.store(out + head + i * kVec);
  }
  for (int i = head + vecs * kVec + threadIdx.x; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(p[i]) * f);
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ TensorTable t, const float* scale) {
  const float f = *scale;
  const uint32_t chunks = t.first[t.tensors];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (f == 1.0f && t.in[i] == t.out[i]) continue;
    const int64_t at = int64_t(c - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(int64_t(kChunk), t.count[i] - at));
    if (t.f32[i])
      scale_chunk(static_cast<const float*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, n, f);
    else
      scale_chunk(static_cast<const __nv_bfloat16*>(t.in[i]) + at, static_cast<__nv_bfloat16*>(t.out[i]) + at, n, f);
  }
}

NormScratch take_norm(Scratch& sc) {
  NormScratch s;
  s.part = sc.take<double>(kMaxBlocks);
  s.carry = sc.take<double>(1);
  s.ticket = sc.take<unsigned>(1);
  s.scale = sc.take<float>(1);
  return s;
}

// Fills the next launch's table from tensor `from` on; returns the tensor after its last.
int64_t fill_table(TensorTable* t, const ClipTensor* list, int64_t num, int64_t from) {
  t->tensors = 0;
  uint64_t chunks = 0;
  int64_t i = from;
  for (; i < num && t->tensors < kTable; ++i) {
    const uint64_t c = static_cast<uint64_t>((list[i].count + kChunk - 1) / kChunk);
    if (!c) continue;
    if (chunks + c > 0xffffffffull) break;
    const int k = t->tensors++;
    t->in[k] = list[i].in;
    t->out[k] = list[i].out;
    t->count[k] = list[i].count;
    t->f32[k] = list[i].dtype == kF32;
    t->first[k] = static_cast<uint32_t>(chunks);
    chunks += c;
  }
  t->first[t->tensors] = static_cast<uint32_t>(chunks);
  return i;
}

}  // namespace

size_t clip_scratch_bytes() {
  Scratch sc;
  take_norm(sc);
  return sc.used();
}

cudaError_t launch_clip(const ClipTensor* list, int64_t num, bool scale, float max_norm, float* norm, Scratch& sc,
                        cudaStream_t st) {
  const NormScratch s = take_norm(sc);
  cudaError_t e = cudaMemsetAsync(s.ticket, 0, sizeof(unsigned), st);
  if (e != cudaSuccess) return e;
  const int most = 4 * ops_sm_count() < kMaxBlocks ? 4 * ops_sm_count() : kMaxBlocks;
  TensorTable t;
  int64_t at = 0;
  bool first = true;
  do {
    const int64_t next = fill_table(&t, list, num, at);
    const uint32_t chunks = t.first[t.tensors];
    const unsigned grid = chunks < 1 ? 1u : (chunks < static_cast<uint32_t>(most) ? chunks : static_cast<unsigned>(most));
    squares_kernel<<<grid, kThreads, 0, st>>>(t, s, first, next >= num, max_norm, norm);
    first = false;
    if (next == at && next < num) return cudaErrorInvalidValue;
    at = next;
  } while (at < num);
  for (at = 0; scale && at < num;) {
    at = fill_table(&t, list, num, at);
    const uint32_t chunks = t.first[t.tensors];
    if (!chunks) continue;
    scale_kernel<<<chunks < static_cast<uint32_t>(most) ? chunks : static_cast<unsigned>(most), kThreads, 0, st>>>(t, s.scale);
  }
  return cudaGetLastError();
}

}  // namespace tk

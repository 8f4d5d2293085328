// The norm of many tensors taken as one vector, and their scaling to a largest
// norm: n = sqrt(sum g^2), g <- g min(1, max_norm / (n + 1e-6)).
//
// The tensors' values are cut into chunks, dealt to the blocks in turn (all
// blocks then read close to each other: one run a block took 45 us where this
// takes 28); the table of tensors goes to the kernel as its parameter, so
// nothing is copied to the device.  A thread sums the squares of one 16-byte
// vector in f32 and adds the vectors' sums in two f32 (a sum and what its
// rounding lost: the card's f64 is slow); the blocks' sums are added in f64 in
// their order.  A vector's sum of four f32 squares is within 2.5 x 2^-24 of it
// (of eight bf16 squares, which are exact, 4.4), and the norm, its own rounding
// included, within 4 x 2^-24, equal values that all round the same way included
// (sums of 128 squares in one f32: 13 x 2^-24 for values of 0.7).  Where the
// f32 squares overflow, or are so small that bits are lost, the chunk is summed
// again in f64, so that this holds for any finite input.
//
// Few values (at most kFewValues) take one launch: a cluster of blocks holds
// them in registers, exchanges its sums through distributed shared memory and
// writes them scaled.  More
// take two: the sums, whose last block forms the norm, and the scaling, which
// goes over the chunks from the last, so that it finds in L2 what was read last.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;            // 16-byte loads of a thread in flight
constexpr int kTable = 640;          // tensors of one launch (the kernel's parameter holds their table)
constexpr int kFewTensors = 48;      // the smaller table of calls with few tensors
constexpr int kMaxBlocks = 2048;
// Bytes at the end of the tensors whose lines L2 is asked to keep from the sums to the scaling (67M bf16 values: 71.7 us
// without, 69.6 with 48 MB, 67.9 with 64, 68.5 with 96).
constexpr int64_t kKeepBytes = int64_t(64) << 20;
constexpr int kCluster = 8;
constexpr int kFewThreads = 512, kFewEach = 16;  // values of a thread, held in registers
constexpr int64_t kFewValues = int64_t(kCluster) * kFewThreads * kFewEach;

template <int N>
struct TensorTable {
  const void* in[N];
  void* out[N];
  int64_t end[N];  // values up to and including the tensor, over the launch
  uint8_t f32[N];
  int tensors;
  int64_t chunk;   // values of a chunk (a multiple of 8)
  int64_t keep;    // chunks at the end whose lines L2 is asked to keep for the scaling
};
struct NormScratch {
  double* part;       // per block of this launch
  double* carry;      // sum of the launches before it
  float* scale;
  unsigned* ticket;   // zero between launches
};

// Calls f(tensor, first value, count) for each tensor's part of values [v0, v1).
template <int N, typename F>
__device__ __forceinline__ void each_part(const TensorTable<N>& t, int64_t v0, int64_t v1, F f) {
  int lo = 0, hi = t.tensors - 1;
  while (lo < hi) {  // the first tensor that ends past v0
    const int mid = (lo + hi) / 2;
    if (t.end[mid] > v0) hi = mid;
    else lo = mid + 1;
  }
  for (; lo < t.tensors && v0 < v1; ++lo) {
    const int64_t first = lo ? t.end[lo - 1] : 0, end = min(t.end[lo], v1);
    if (end > v0) f(lo, v0 - first, end - v0);
    v0 = max(v0, end);
  }
}

// L2's policy for lines that are read again soon.
__device__ __forceinline__ uint64_t l2_evict_last_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ uint4 load_hint(const uint4* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "l"(policy));
  return v;
}
// Goes over the block's values of [p, p + n), from the end when BACKWARD: whole
// 16-byte vectors (aligned to those of p) kAhead at a time through `vec(values,
// place)`, single values at the ends through `one(value, place)`.
template <typename T, bool BACKWARD, typename V, typename O>
__device__ __forceinline__ void each_value(const T* p, int64_t n, uint64_t policy, V vec, O one) {
  constexpr int kVec = 16 / sizeof(T);
  const int64_t head = min(n, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int64_t(sizeof(T)));
  const int64_t vecs = (n - head) / kVec;
  for (int64_t i = threadIdx.x; i < head; i += kThreads) one(to_f32(p[i]), i);
  const int64_t steps = vecs / (kThreads * kAhead);
  const uint4* q = reinterpret_cast<const uint4*>(p + head) + threadIdx.x;
  auto rest = [&] {  // less than a whole step, at the end
    for (int64_t i = steps * (kThreads * kAhead) + threadIdx.x; i < vecs; i += kThreads) {
      Vec<T, kVec> v;
      v.set(load_hint(q + (i - threadIdx.x), policy));
      vec(v, head + i * kVec);
    }
  };
  if (BACKWARD) rest();
#pragma unroll 1
  for (int64_t s = 0; s < steps; ++s) {
    const int64_t i0 = (BACKWARD ? steps - 1 - s : s) * (kThreads * kAhead);
    uint4 raw[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) raw[a] = load_hint(q + i0 + a * kThreads, policy);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      Vec<T, kVec> v;
      v.set(raw[a]);
      vec(v, head + (i0 + a * kThreads + threadIdx.x) * kVec);
    }
  }
  if (!BACKWARD) rest();
  for (int64_t i = head + vecs * kVec + threadIdx.x; i < n; i += kThreads) one(to_f32(p[i]), i);
}

template <typename T>
__device__ __noinline__ double part_squares_wide(const T* p, int64_t n, uint64_t policy) {
  constexpr int kVec = 16 / sizeof(T);
  double wide = 0.0;
  each_value<T, false>(
      p, n, policy,
      [&](const Vec<T, kVec>& v, int64_t) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) wide += static_cast<double>(v.v[c]) * v.v[c];
      },
      [&](float v, int64_t) { wide += static_cast<double>(v) * v; });
  return wide;
}

// A sum in two f32: the rounded sum, and what the roundings lost.
struct TwoSum {
  float hi, lo;
  __device__ __forceinline__ void add(float v) {
    const float s = hi + v, b = s - hi;
    lo += (hi - (s - b)) + (v - b);
    hi = s;
  }
};
struct Squares {
  TwoSum sum{0.0f, 0.0f};
  double wide = 0.0;  // what f32 could not hold
};

template <typename T>
__device__ __forceinline__ void part_squares(const T* p, int64_t n, uint64_t policy, Squares* to) {
  constexpr int kVec = 16 / sizeof(T);
  TwoSum sum{0.0f, 0.0f};
  float most = 0.0f;
  each_value<T, false>(
      p, n, policy,
      [&](const Vec<T, kVec>& v, int64_t) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          s = fmaf(v.v[c], v.v[c], s);
          most = fmaxf(most, fabsf(v.v[c]));
        }
        sum.add(s);
      },
      [&](float v, int64_t) {
        sum.add(v * v);
        most = fmaxf(most, fabsf(v));
      });
  // f32 squares neither overflow nor lose bits between these (a block's sum of them stays below 2^127 for any tensor
  // that fits the card); zeros stay what they are, NaN and infinities go on through f64
  if (most == 0.0f && sum.hi == 0.0f) return;
  if (most > 1e-15f && most < 1e12f && sum.hi < INFINITY) {
    to->sum.add(sum.hi);
    to->sum.lo += sum.lo;
  } else {
    to->wide += part_squares_wide(p, n, policy);
  }
}

template <int N>
__device__ __forceinline__ void chunk_squares(const TensorTable<N>& t, int64_t chunk, uint64_t policy, Squares* to) {
  const int64_t v0 = chunk * t.chunk, v1 = min(v0 + t.chunk, t.end[t.tensors - 1]);
  each_part(t, v0, v1, [&](int i, int64_t at, int64_t n) {
    if (t.f32[i]) part_squares(static_cast<const float*>(t.in[i]) + at, n, policy, to);
    else part_squares(static_cast<const __nv_bfloat16*>(t.in[i]) + at, n, policy, to);
  });
}
template <int N>
__device__ __forceinline__ int64_t chunks_of(const TensorTable<N>& t) {
  return t.tensors ? (t.end[t.tensors - 1] + t.chunk - 1) / t.chunk : 0;
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
__device__ __forceinline__ float scale_of(float norm, float max_norm) {
  const float f = max_norm / (norm + 1e-6f);
  return f > 1.0f ? 1.0f : f;  // (NaN stays NaN)
}

template <typename T>
__device__ __forceinline__ void scale_part(const T* p, T* out, int64_t n, uint64_t policy, float f) {
  constexpr int kVec = 16 / sizeof(T);
  const bool apart = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0;
  each_value<T, true>(
      p, n, policy,
      [&](const Vec<T, kVec>& v, int64_t at) {
        Vec<T, kVec> o;
#pragma unroll
        for (int c = 0; c < kVec; ++c) o.v[c] = v.v[c] * f;
        if (apart) {
#pragma unroll
          for (int c = 0; c < kVec; ++c) out[at + c] = from_f32<T>(o.v[c]);
        } else {
          __stcs(reinterpret_cast<uint4*>(out + at), o.pack());
        }
      },
      [&](float v, int64_t at) { out[at] = from_f32<T>(v * f); });
}
template <int N>
__device__ __forceinline__ void scale_chunk(const TensorTable<N>& t, int64_t chunk, uint64_t policy, float f) {
  const int64_t v0 = chunk * t.chunk, v1 = min(v0 + t.chunk, t.end[t.tensors - 1]);
  each_part(t, v0, v1, [&](int i, int64_t at, int64_t n) {
    if (f == 1.0f && t.in[i] == t.out[i]) return;
    if (t.f32[i])
      scale_part(static_cast<const float*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, n, policy, f);
    else
      scale_part(static_cast<const __nv_bfloat16*>(t.in[i]) + at, static_cast<__nv_bfloat16*>(t.out[i]) + at, n, policy, f);
  });
}

template <int N>
__global__ void __launch_bounds__(kThreads, 8) squares_kernel(const __grid_constant__ TensorTable<N> t, NormScratch s, bool first,
                                                           bool finish, float max_norm, float* norm) {
  __shared__ double shared[kThreads / 32];
  __shared__ bool last;
  grid_dependency_wait();
  grid_launch_dependents();
  Squares mine;
  const uint64_t first_out = l2_evict_first_policy(), last_out = l2_evict_last_policy();
  for (int64_t c = blockIdx.x; c < chunks_of(t); c += gridDim.x) chunk_squares(t, c, c < chunks_of(t) - t.keep ? first_out : last_out, &mine);
  // the warps' sums in two f32, the block's in f64
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float hi = __shfl_xor_sync(~0u, mine.sum.hi, o), lo = __shfl_xor_sync(~0u, mine.sum.lo, o);
    mine.sum.add(hi);
    mine.sum.lo += lo;
  }
  double sum = 0.0;
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = static_cast<double>(mine.sum.hi) + mine.sum.lo;
  const bool any_wide = __syncthreads_or(mine.wide != 0.0);  // (NaN too)
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) sum += shared[w];
  if (any_wide) {
    __syncthreads();
    sum += block_sum(mine.wide, shared);
  }
  if (threadIdx.x == 0) {
    s.part[blockIdx.x] = sum;
    __threadfence();
    last = atomicInc(s.ticket, gridDim.x - 1) == gridDim.x - 1;  // (back to 0 for the next launch)
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
    if (finish) {
      const float n = static_cast<float>(sqrt(all));
      *norm = n;
      *s.scale = scale_of(n, max_norm);
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 8) scale_kernel(const __grid_constant__ TensorTable<N> t, const float* scale) {
  grid_dependency_wait();
  grid_launch_dependents();
  const float f = *scale;
  const uint64_t policy = l2_evict_first_policy();
  for (int64_t c = chunks_of(t) - 1 - blockIdx.x; c >= 0; c -= gridDim.x) scale_chunk(t, c, policy, f);
}

// Norm and scaling of few values by one cluster.  Values are dealt to threads
// one at a time, whatever tensor they lie in, all loads of a thread in flight.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kFewThreads)
    clip_few_kernel(const __grid_constant__ TensorTable<kFewTensors> t, bool scale, float max_norm, float* norm) {
  __shared__ double shared[kFewThreads / 32];
  __shared__ double sums[kCluster];
  __shared__ int64_t ends[kFewTensors];
  __shared__ const void* ins[kFewTensors];
  if (threadIdx.x < t.tensors) {
    ends[threadIdx.x] = t.end[threadIdx.x];
    ins[threadIdx.x] = t.in[threadIdx.x];
  }
  __syncthreads();
  // (every block of the cluster has started before another writes to its memory)
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_launch_dependents();
  const int values = t.tensors ? static_cast<int>(t.end[t.tensors - 1]) : 0;
  float v[kFewEach];
  int where[kFewEach];  // tensor, or -1
#pragma unroll
  for (int e = 0; e < kFewEach; ++e) {
    const int at = (e * kCluster + static_cast<int>(blockIdx.x)) * kFewThreads + static_cast<int>(threadIdx.x);
    v[e] = 0.0f;
    where[e] = -1;
    if (at < values) {
      int lo = 0, hi = t.tensors - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ends[mid] > at) hi = mid;
        else lo = mid + 1;
      }
      const int64_t i = at - (lo ? ends[lo - 1] : 0);
      v[e] = t.f32[lo] ? static_cast<const float*>(ins[lo])[i] : to_f32(static_cast<const __nv_bfloat16*>(ins[lo])[i]);
      where[e] = lo;
    }
  }
  // in two f32 over a warp, then f64; all in f64 where the squares leave f32 or lose bits (the card's f64 is slow)
  TwoSum two{0.0f, 0.0f};
  float most = 0.0f;
#pragma unroll
  for (int e = 0; e < kFewEach; ++e) {
    two.add(v[e] * v[e]);
    most = fmaxf(most, fabsf(v[e]));
  }
  double sum;
  if (__all_sync(~0u, most == 0.0f || !(most < INFINITY) || (most > 1e-15f && most < 1e17f))) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float hi = __shfl_xor_sync(~0u, two.hi, o), lo = __shfl_xor_sync(~0u, two.lo, o);
      two.add(hi);
      two.lo += lo;
    }
    // (an infinity or NaN in hi leaves NaN in lo)
    sum = fabsf(two.hi) < INFINITY ? static_cast<double>(two.hi) + two.lo : static_cast<double>(two.hi);
  } else {
    sum = 0.0;
#pragma unroll
    for (int e = 0; e < kFewEach; ++e) sum += static_cast<double>(v[e]) * v[e];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  }
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x < kCluster) {  // this block's sum to every block of the cluster
    sum = 0.0;
    for (int w = 0; w < kFewThreads / 32; ++w) sum += shared[w];
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(&sums[blockIdx.x])), "r"(threadIdx.x));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(sum) : "memory");
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  double all = 0.0;
#pragma unroll
  for (int b = 0; b < kCluster; ++b) all += sums[b];
  const float n = static_cast<float>(sqrt(all));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  if (!scale) return;
  const float f = scale_of(n, max_norm);
#pragma unroll
  for (int e = 0; e < kFewEach; ++e) {
    if (where[e] < 0) continue;
    const int lo = where[e];
    const int at = (e * kCluster + static_cast<int>(blockIdx.x)) * kFewThreads + static_cast<int>(threadIdx.x);
    const int64_t i = at - (lo ? ends[lo - 1] : 0);
    if (t.f32[lo]) static_cast<float*>(t.out[lo])[i] = v[e] * f;
    else static_cast<__nv_bfloat16*>(t.out[lo])[i] = from_f32<__nv_bfloat16>(v[e] * f);
  }
}

NormScratch take_norm(Scratch& sc) {
  NormScratch s;
  s.part = sc.take<double>(kMaxBlocks);
  s.carry = sc.take<double>(1);
  s.scale = sc.take<float>(1);
  s.ticket = nullptr;
  return s;
}

// Fills the next launch's table from tensor `from` on; returns the tensor after its last.
template <int N>
int64_t fill_table(TensorTable<N>* t, const ClipTensor* list, int64_t num, int64_t from) {
  t->tensors = 0;
  int64_t values = 0, i = from;
  for (; i < num && t->tensors < N; ++i) {
    if (!list[i].count) continue;
    const int k = t->tensors++;
    values += list[i].count;
    t->in[k] = list[i].in;
    t->out[k] = list[i].out;
    t->end[k] = values;
    t->f32[k] = list[i].dtype == kF32;
  }
  return i;
}
// Blocks for the table's chunks: as many as fit at once.
template <int N>
unsigned cut_chunks(TensorTable<N>* t, int64_t most, bool scale) {
  const int64_t values = t->tensors ? t->end[t->tensors - 1] : 0;
  int64_t bytes = 0;
  for (int i = 0; i < t->tensors; ++i) bytes += (t->end[i] - (i ? t->end[i - 1] : 0)) * (t->f32[i] ? 4 : 2);
  t->chunk = kThreads * kAhead * 32;
  t->keep = scale && bytes ? static_cast<int64_t>(static_cast<double>(kKeepBytes) / bytes * values / t->chunk) : 0;
  const int64_t blocks = (values + t->chunk - 1) / t->chunk;
  return static_cast<unsigned>(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

template <int N>
cudaError_t launch_many(const ClipTensor* list, int64_t num, bool scale, float max_norm, float* norm, const NormScratch& s,
                        cudaStream_t st) {
  // as many blocks as fit at once, so that they end near the same time
  static PerDevice fits;
  std::atomic<int>* known = fits.here();
  int each = known ? known->load() : 0;
  if (!each) {
    int a = 0, b = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&a, squares_kernel<N>, kThreads, 0);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, scale_kernel<N>, kThreads, 0);
    if (e != cudaSuccess) return e;
    a = a < b ? a : b;
    each = a < 1 ? 1 : a;
    if (known) *known = each;
  }
  const int64_t fit = int64_t(each) * ops_sm_count(), most = fit < kMaxBlocks ? fit : kMaxBlocks;
  TensorTable<N> t;
  int64_t at = 0;
  bool first = true;
  int launches = 0;
  do {
    ++launches;
    at = fill_table(&t, list, num, at);
    const cudaError_t e = launch_after(squares_kernel<N>, cut_chunks(&t, most, scale), kThreads, 0, st, t, s, first, at >= num, max_norm, norm);
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < num);
  if (!scale) return cudaSuccess;
  at = 0;
  do {
    if (launches > 1) at = fill_table(&t, list, num, at);
    if (t.tensors) {
      const unsigned blocks = cut_chunks(&t, most, scale);
      const cudaError_t e = launch_after(scale_kernel<N>, blocks, kThreads, 0, st, t, static_cast<const float*>(s.scale));
      if (e != cudaSuccess) return e;
    }
  } while (launches > 1 && at < num);
  return cudaSuccess;
}

}  // namespace

size_t clip_scratch_bytes() {
  Scratch sc;
  take_norm(sc);
  return sc.used();
}

cudaError_t launch_clip(const ClipTensor* list, int64_t num, bool scale, float max_norm, float* norm, const Words& words,
                        Scratch& sc, cudaStream_t st) {
  NormScratch s = take_norm(sc);
  s.ticket = reinterpret_cast<unsigned*>(words.at) + 32;
  int64_t values = 0, tensors = 0;
  for (int64_t i = 0; i < num; ++i) {
    values += list[i].count;
    tensors += list[i].count > 0;
  }
  if (tensors <= kFewTensors && values <= kFewValues) {
    TensorTable<kFewTensors> t;
    fill_table(&t, list, num, 0);
    return launch_after(clip_few_kernel, unsigned(kCluster), kFewThreads, 0, st, t, scale, max_norm, norm);
  }
  return tensors <= kFewTensors ? launch_many<kFewTensors>(list, num, scale, max_norm, norm, s, st)
                                : launch_many<kTable>(list, num, scale, max_norm, norm, s, st);
}

}  // namespace tk

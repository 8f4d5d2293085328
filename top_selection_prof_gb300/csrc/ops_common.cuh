// Device helpers of the operators around the selection: conversions between
// the storage types and f32, vector loads, activations.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ops.h"

namespace tk {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Rounded to nearest even (the one rounding of each result).
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two f32 side by side in a register pair, multiplied and added in one instruction.
struct Pair {
  uint64_t u;
  __device__ __forceinline__ static Pair of(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.u) : "f"(a), "f"(b));
    return p;
  }
  __device__ __forceinline__ void get(float* a, float* b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(u)); }
  __device__ __forceinline__ void fma(Pair a, Pair b) { asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(u) : "l"(a.u), "l"(b.u)); }
};

// 16 bytes from global to shared memory without passing through registers; the
// thread's copies are in place after copy_async_wait().
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// VEC values: 16 bytes, or one f32; one bf16 (which has no such copy) goes through a register.
template <int VEC, typename T>
__device__ __forceinline__ void copy_async(T* dst, const T* src) {
  if constexpr (VEC > 1) copy_async16(dst, src);
  else if constexpr (sizeof(T) == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
  else *dst = __ldg(src);
}
// Groups of copies, done in their order: all but the last N are in place after copy_async_wait_group<N>().
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// VEC consecutive values as they are stored.
template <typename T, int VEC>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load_nc(const T* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  // Values 2 i and 2 i + 1 as f32.
  __device__ __forceinline__ Pair pair(int i) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) return Pair::of(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    return Pair::of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <typename T>
struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void load_nc(const T* p) { u = __ldg(p); }
  __device__ __forceinline__ void load(const T* p) { u = *p; }
  __device__ __forceinline__ void clear() { u = from_f32<T>(0.0f); }
};

// VEC consecutive values as f32: one 16-byte access when VEC values fill 16
// bytes (p then 16-byte aligned), one value when VEC == 1.
template <typename T, int VEC>
struct Vec {
  static_assert(VEC == 1 || VEC * sizeof(T) == 16, "one value or 16 bytes");
  static constexpr int kWide = VEC;
  float v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1) {
      v[0] = to_f32(*p);
    } else {
      set(*reinterpret_cast<const uint4*>(p));
    }
  }
  // (past the L1: what another block wrote in this launch)
  __device__ __forceinline__ void load_cg(const T* p) {
    if constexpr (VEC == 1) {
      v[0] = to_f32(__ldcg(p));
    } else {
      set(__ldcg(reinterpret_cast<const uint4*>(p)));
    }
  }
  __device__ __forceinline__ void load_nc(const T* p) {
    if constexpr (VEC == 1) {
      v[0] = to_f32(__ldg(p));
    } else {
      set(__ldg(reinterpret_cast<const uint4*>(p)));
    }
  }
  __device__ __forceinline__ void set(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        v[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
      }
    }
  }
  __device__ __forceinline__ uint4 pack() const {
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void set_raw(const Raw<T, VEC>& r) {
    if constexpr (VEC == 1) v[0] = to_f32(r.u);
    else set(r.u);
  }
  // (written once and not read again here)
  __device__ __forceinline__ void store_stream(T* p) const {
    if constexpr (VEC == 1) *p = from_f32<T>(v[0]);
    else __stcs(reinterpret_cast<uint4*>(p), pack());
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 1) {
      *p = from_f32<T>(v[0]);
    } else {
      *reinterpret_cast<uint4*>(p) = pack();
    }
  }
};

// What an f32 product by parts does with operands that are marked.  The third part of a value below kSmall would leave
// bf16's range (2^-133): such an operand is scaled by kScale, unless a value of kLarge or more in either could then
// overflow a sum (k < 2^31: 2^31 (2^32 kScale)^2 = 2^127); then, as with an infinity, the product goes to the CUDA cores.
constexpr float kSmall = 0x1p-110f, kLarge = 0x1p32f, kScale = 0x1p16f, kUnscale = 0x1p-16f;
struct PartsPlan {
  bool cores;             // made on the CUDA cores
  bool scale_a, scale_b;
};
__device__ __forceinline__ PartsPlan parts_plan(const int* marks, int call) {
  const bool a = marks[kMarkSmallA] == call, b = marks[kMarkSmallB] == call;
  const bool cores = marks[kMarkOther] == call || ((a || b) && marks[kMarkLarge] == call);
  return {cores, a && !cores, b && !cores};
}

// Launches a kernel that calls grid_dependency_wait() before it touches memory:
// it may start, and set itself up, while the grid before it in the stream ends.
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// act(z) and act'(z), for results of type T.  relu(NaN) = NaN and relu'(NaN) =
// 0.  gelu is the exact form z Phi(z), silu z / (1 + e^-z); both are 0 at -inf
// (where their formulas meet inf x 0) and z at inf.
//
// f32 results take CUDA's erfcf and expf (Phi(z) = erfc(-z / sqrt 2) / 2: with 1 + erf, what is left of the sum at z = -5 is
// off by 4 %).  bf16 results, whose own rounding is
// 2^-9, take the hardware's exponential and reciprocal (2^-22) and
//   Phi(-a) = e^(-a^2/2) t (c1 + c2 t + ... + c6 t^5),  t = 1 / (1 + 0.31 a),  a >= 0,
// the coefficients fitted (weighted least squares, reweighted towards the
// largest error) to e^(a^2/2) Phi(-a) on [0, 14] with a relative error of at
// most 4.8e-6: with erff the epilogue of 4096 x 512 x 65536 took 695 us where
// the product takes 180.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Phi(-a) for 0 <= a <= 16, and e = e^(-a^2/2).
__device__ __forceinline__ float fast_upper_tail(float a, float* e) {
  const float t = fast_rcp(fmaf(0.31f, a, 1.0f));
  *e = fast_exp2(a * a * -0.72134752f);
  float s = fmaf(t, -0.07392814f, 0.18044704f);
  s = fmaf(s, t, 0.015749037f);
  s = fmaf(s, t, 0.13342702f);
  s = fmaf(s, t, 0.12044213f);
  s = fmaf(s, t, 0.12386061f);
  return s * t * *e;
}
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }
__device__ __forceinline__ float relu(float z) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
  return y;
}

// s = 1 / (1 + e^-z) and t = 1 - s, both from e^-|z|: neither cancels, nor overflows below z = -88, where z s is still 1e-36.
template <typename T>
__device__ __forceinline__ void logistic(float z, float* s, float* t) {
  const float a = fabsf(z);
  const float e = sizeof(T) == 2 ? fast_exp2(a * -1.44269504f) : expf(-a);
  const float r = sizeof(T) == 2 ? fast_rcp(1.0f + e) : 1.0f / (1.0f + e);
  *s = z < 0.0f ? e * r : r;
  *t = z < 0.0f ? r : e * r;
}

template <typename T>
__device__ __forceinline__ float act_value(float z, int act) {
  constexpr bool kFast = sizeof(T) == 2;
  switch (act) {
    case kActRelu: return relu(z);
    case kActGelu:
      if constexpr (kFast) {
        float a = fabsf(z), e;
        a = a > 16.0f ? 16.0f : a;  // (NaN stays)
        const float low = (z < 0.0f ? -a : a) * fast_upper_tail(a, &e);
        return z >= 0.0f ? z - low : low;
      }
      return z == -INFINITY ? 0.0f : z * normal_cdf(z);
    case kActSilu: {
      float s, t;
      logistic<T>(z, &s, &t);
      return z == -INFINITY ? 0.0f : z * s;
    }
    default: return z;
  }
}
template <typename T>
__device__ __forceinline__ float act_slope(float z, int act) {
  constexpr bool kFast = sizeof(T) == 2;
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : 0.0f;
    case kActGelu:
      if (fabsf(z) > 16.0f) return z > 0.0f ? 1.0f : 0.0f;
      if constexpr (kFast) {
        float e;
        const float q = fast_upper_tail(fabsf(z), &e);
        return fmaf(z * e, 0.39894228f, z < 0.0f ? q : 1.0f - q);
      }
      return normal_cdf(z) + z * expf(-0.5f * z * z) * 0.3989422804014327f;
    case kActSilu: {
      if (fabsf(z) == INFINITY) return z > 0.0f ? 1.0f : 0.0f;
      float s, t;
      logistic<T>(z, &s, &t);
      return s * (1.0f + z * t);
    }
    default: return 1.0f;
  }
}

}  // namespace tk

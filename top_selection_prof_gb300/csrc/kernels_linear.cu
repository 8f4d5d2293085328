// Matrix products with a fused epilogue, and the pass that prepares their
// gradients: c = act(a b^T + bias) + residual for the linear layer, and the
// plain products of its backward pass, over operands of either order.
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

// ---------------------------------------------------------------------------
// Products on the CUDA cores.  One block of 256 threads makes a 128 x 128 tile
// of c from 16-deep slices in shared memory, 8 x 8 results a thread in
// registers, every product and sum in f32.
// ---------------------------------------------------------------------------
constexpr int kTile = 128, kDeep = 16, kSimtThreads = 256;
constexpr int kTilePad = kTile + 4;

template <typename T>
struct SimtParams {
  const T* a;
  const T* b;
  int64_t lda, ldb;
  bool a_k_inner, b_k_inner;
  int64_t m, n, k;
  const T* bias;
  const T* residual;
  int64_t ldr;
  int act;
  T* c;
  int64_t ldc;
  T* pre;
  int64_t ldp;
  int64_t tiles_n;
};

// A kDeep x kTile slice of an operand into shared memory, as f32, zeros outside it.
template <typename T>
__device__ __forceinline__ void load_slice(float (&dst)[kDeep][kTilePad], const T* p, int64_t ld, bool k_inner,
                                           int64_t i0, int64_t rows, int64_t k0, int64_t k) {
  constexpr int kEach = kTile * kDeep / kSimtThreads;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int at = e * kSimtThreads + static_cast<int>(threadIdx.x);
    int i, j;
    if (k_inner) {
      i = at / kDeep;
      j = at % kDeep;
    } else {
      i = at % kTile;
      j = at / kTile;
    }
    const int64_t gi = i0 + i, gk = k0 + j;
    float v = 0.0f;
    if (gi < rows && gk < k) v = to_f32(k_inner ? p[gi * ld + gk] : p[gk * ld + gi]);
    dst[j][i] = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(kSimtThreads) simt_product_kernel(const SimtParams<T> p) {
  __shared__ float as[kDeep][kTilePad], bs[kDeep][kTilePad];
  const int64_t m0 = (blockIdx.x / p.tiles_n) * kTile, n0 = (blockIdx.x % p.tiles_n) * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[8][8] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += kDeep) {
    load_slice(as, p.a, p.lda, p.a_k_inner, m0, p.m, k0, p.k);
    load_slice(bs, p.b, p.ldb, p.b_k_inner, n0, p.n, k0, p.k);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      float av[8], bv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) av[i] = as[j][(i / 4) * 64 + ty * 4 + i % 4];
#pragma unroll
      for (int i = 0; i < 8; ++i) bv[i] = bs[j][(i / 4) * 64 + tx * 4 + i % 4];
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t i = m0 + (r / 4) * 64 + ty * 4 + r % 4;
    if (i >= p.m) continue;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int64_t j = n0 + (c / 4) * 64 + tx * 4 + c % 4;
      if (j >= p.n) continue;
      float z = acc[r][c] + (p.bias ? to_f32(p.bias[j]) : 0.0f);
      if (p.pre) p.pre[i * p.ldp + j] = from_f32<T>(z);
      z = act_value(z, p.act);
      if (p.residual) z += to_f32(p.residual[i * p.ldr + j]);
      p.c[i * p.ldc + j] = from_f32<T>(z);
    }
  }
}

template <typename T>
cudaError_t launch_simt(const Product& g, cudaStream_t st) {
  SimtParams<T> p;
  p.a = static_cast<const T*>(g.a.p);
  p.b = static_cast<const T*>(g.b.p);
  p.lda = g.a.ld;
  p.ldb = g.b.ld;
  p.a_k_inner = g.a.k_inner;
  p.b_k_inner = g.b.k_inner;
  p.m = g.m;
  p.n = g.n;
  p.k = g.k;
  p.bias = static_cast<const T*>(g.bias);
  p.residual = static_cast<const T*>(g.residual);
  p.ldr = g.ldr;
  p.act = g.act;
  p.c = static_cast<T*>(g.c);
  p.ldc = g.ldc;
  p.pre = static_cast<T*>(g.pre);
  p.ldp = g.ldp;
  p.tiles_n = (g.n + kTile - 1) / kTile;
  const int64_t tiles = p.tiles_n * ((g.m + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  simt_product_kernel<T><<<static_cast<unsigned>(tiles), kSimtThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// dz = dy act'(pre) and its column sums.  A block takes 64 columns x
// kSumRows rows (8 rows of threads); a column's partial sums go to part[block
// row][column] and are added in that order by the second kernel.
// ---------------------------------------------------------------------------
constexpr int kSumCols = 64, kSumThreads = 256, kSumRows = 256;

template <typename T>
__global__ void __launch_bounds__(kSumThreads) slope_sums_kernel(const SlopeSums s) {
  const T* dy = static_cast<const T*>(s.dy);
  const T* pre = static_cast<const T*>(s.pre);
  T* dz = static_cast<T*>(s.dz);
  __shared__ float sums[kSumThreads / kSumCols][kSumCols];
  const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
  const int64_t col_blocks = (s.n + kSumCols - 1) / kSumCols;
  const int64_t rb = blockIdx.x / col_blocks;
  const int64_t j = (blockIdx.x % col_blocks) * kSumCols + tx;
  const int64_t r1 = min(s.rows, (rb + 1) * kSumRows);
  float acc = 0.0f;
  if (j < s.n) {
    for (int64_t r = rb * kSumRows + ty; r < r1; r += kSumThreads / kSumCols) {
      float v = to_f32(dy[r * s.lddy + j]);
      if (s.act != kActNone) {
        v *= act_slope(to_f32(pre[r * s.ldp + j]), s.act);
        if (dz) dz[r * s.n + j] = from_f32<T>(v);
      }
      acc += v;
    }
  }
  sums[ty][tx] = acc;
  __syncthreads();
  if (s.dbias && ty == 0 && j < s.n) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumThreads / kSumCols; ++i) t += sums[i][tx];
    s.part[rb * s.n + j] = t;
  }
}

template <typename T>
__global__ void sum_parts_kernel(const float* part, int64_t parts, int64_t n, T* out) {
  const int64_t j = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (j >= n) return;
  float t = 0.0f;
  for (int64_t i = 0; i < parts; ++i) t += part[i * n + j];
  out[j] = from_f32<T>(t);
}

template <typename T>
cudaError_t launch_slope_sums_t(const SlopeSums& s, cudaStream_t st) {
  const int64_t parts = slope_sums_parts(s.rows, s.n);
  const int64_t blocks = parts * ((s.n + kSumCols - 1) / kSumCols);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  slope_sums_kernel<T><<<static_cast<unsigned>(blocks), kSumThreads, 0, st>>>(s);
  if (s.dbias)
    sum_parts_kernel<T><<<static_cast<unsigned>((s.n + 127) / 128), 128, 0, st>>>(s.part, parts, s.n,
                                                                                  static_cast<T*>(s.dbias));
  return cudaGetLastError();
}

}  // namespace

int64_t slope_sums_parts(int64_t rows, int64_t) { return (rows + kSumRows - 1) / kSumRows; }

cudaError_t launch_slope_sums(const SlopeSums& s, cudaStream_t st) {
  return s.dtype == kF32 ? launch_slope_sums_t<float>(s, st) : launch_slope_sums_t<__nv_bfloat16>(s, st);
}

size_t product_scratch_bytes(const Product& g) { return g.dtype == kF32 ? 0 : mma_scratch_bytes(g); }

cudaError_t launch_product(const Product& g, Scratch& sc, int* words, cudaStream_t st) {
  return g.dtype == kF32 ? launch_simt<float>(g, st) : launch_mma(g, sc, words, st);
}

}  // namespace tk

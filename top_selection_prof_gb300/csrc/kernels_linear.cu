// Matrix products with a fused epilogue, and the pass that prepares their
// gradients: c = act(a b^T + bias) + residual for the linear layer, and the
// plain products of its backward pass, over operands of either order.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

// ---------------------------------------------------------------------------
// f32 products on the CUDA cores: what runs in the tensor cores' place when an
// operand holds an infinity or NaN (their three-part form has no such
// values), or values of both ends of f32's range meet.  One block of 256
// threads makes a 128 x 128 tile of c from 16-deep slices in shared memory,
// 8 x 8 results a thread in registers, every product and sum in f32.  It does
// nothing, at the cost of its launch, unless the operands' split left this
// call's marks.
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
  const int* marks;  // the product is made only where these say so for `call`
  int call;
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
  grid_dependency_wait();
  grid_launch_dependents();
  if (!parts_plan(p.marks, p.call).cores) return;
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
      z = act_value<T>(z, p.act);
      if (p.residual) z += to_f32(p.residual[i * p.ldr + j]);
      p.c[i * p.ldc + j] = from_f32<T>(z);
    }
  }
}

cudaError_t launch_simt_t(const Product& g, const int* marks, int call, cudaStream_t st) {
  using T = float;
  SimtParams<T> p;
  p.marks = marks;
  p.call = call;
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
  if (tiles > INT32_MAX) return cudaErrorNotSupported;
  return launch_after(simt_product_kernel<T>, static_cast<unsigned>(tiles), kSimtThreads, 0, st, p);
}

// ---------------------------------------------------------------------------
// Products of few rows: y = act(x w^T + bias) + residual, one pass over w for
// each R <= 8 rows of x.  A warp takes kFewCols rows of w (or a KS-th of their
// length), 16 bytes of each a lane and step, and keeps kFewCols x R sums, of
// even and odd k side by side; the lanes' sums are added by exchanging halves.
// ---------------------------------------------------------------------------
constexpr int kFewCols = 4, kFewWarps = 8;
// Threads an SM holds at once, which bounds the registers of each.  Blocks of four warps where a thread has many: 8 rows of
// f32 take 75 us at 4096 -> 16384 with 12 warps an SM, 91 with 8; 1 row 43 with 32 and 55 with 24.  Two rows
// have no variant of their own (36 us at 4096 -> 16384 bf16, 29 as four), nor two to four off 16-byte boundaries (4097 ->
// 16384 f32: 86 us, 69 as eight); one such row keeps eight steps of w on their way (bf16: 38 us, 98 with four).
constexpr int few_resident(int vec, int rows) {
  return vec == 1 ? 512 : rows == 1 ? 1024 : rows == 4 ? 512 : 384;
}

template <typename T>
struct FewParams {
  const T* x;
  const T* w;
  int64_t ldx, ldw, rows, n, k, k_run;  // k_run: length of one KS-th
  const T* bias;
  const T* residual;
  int64_t ldr;
  int act;
  T* y;
  int64_t ldy;
  T* pre;
  int64_t ldp;
};

template <typename T, int VEC, int R>
__global__ void __launch_bounds__(few_resident(VEC, R)) few_rows_kernel(const FewParams<T> p, int ks) {
  constexpr int kSums = kFewCols * R;
  __shared__ float sums[kFewWarps][kSums];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = int(blockDim.x) / 32 / ks, group = warp / ks, part = warp % ks;
  const unsigned passes = static_cast<unsigned>((p.rows + R - 1) / R);  // side by side, so that w is in L2 for all but the first
  const int64_t n0 = (int64_t(blockIdx.x / passes) * groups + group) * kFewCols;
  const int64_t r0 = blockIdx.x % passes * R;
  float acc[kSums] = {};
  const T* wp[kFewCols];
#pragma unroll
  for (int c = 0; c < kFewCols; ++c) wp[c] = p.w + min(n0 + c, p.n - 1) * p.ldw;
  const T* xp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) xp[r] = p.x + min(r0 + r, p.rows - 1) * p.ldx;
  const int64_t k1 = min(p.k, (part + 1) * p.k_run);
  if constexpr (VEC == 1) {
#pragma unroll (R == 1 ? 8 : 4)
    for (int64_t k = part * p.k_run + lane; k < k1; k += 32) {
      float wv[kFewCols];
#pragma unroll
      for (int c = 0; c < kFewCols; ++c) wv[c] = to_f32(__ldg(wp[c] + k));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float xv = to_f32(__ldg(xp[r] + k));
#pragma unroll
        for (int c = 0; c < kFewCols; ++c) acc[c * R + r] = fmaf(wv[c], xv, acc[c * R + r]);
      }
    }
  } else {
    Pair two[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) two[i] = Pair::of(0.0f, 0.0f);
    // the next step's part of w on its way
    Raw<T, VEC> next[kFewCols];
    int64_t k = part * p.k_run + lane * VEC;
#pragma unroll
    for (int c = 0; c < kFewCols; ++c)
      if (k < k1) next[c].load_nc(wp[c] + k);
#pragma unroll 1
    for (; k < k1; k += 32 * VEC) {
      Pair wv[kFewCols][VEC / 2];
#pragma unroll
      for (int c = 0; c < kFewCols; ++c) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) wv[c][i] = next[c].pair(i);
        if (k + 32 * VEC < k1) next[c].load_nc(wp[c] + k + 32 * VEC);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Raw<T, VEC> xr;
        xr.load_nc(xp[r] + k);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const Pair xv = xr.pair(i);
#pragma unroll
          for (int c = 0; c < kFewCols; ++c) two[c * R + r].fma(wv[c][i], xv);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      float lo, hi;
      two[i].get(&lo, &hi);
      acc[i] = lo + hi;
    }
  }
  // halves exchanged until a lane holds one sum: sum i in the lanes whose high bits say i
  int o = 16;
#pragma unroll
  for (int h = kSums / 2; h >= 1; h /= 2) {
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const bool high = lane & o;
      const float give = high ? acc[i] : acc[i + h];
      acc[i] = (high ? acc[i + h] : acc[i]) + __shfl_xor_sync(~0u, give, o);
    }
    o /= 2;
  }
  for (; o; o /= 2) acc[0] += __shfl_xor_sync(~0u, acc[0], o);
  constexpr int kLanes = 32 / kSums;  // lanes that hold the same sum
  if (lane % kLanes == 0) sums[warp][lane / kLanes] = acc[0];
  __syncthreads();
  // each group's first lanes finish its sums, the parts in their order
  if (part != 0 || lane >= kSums) return;
  float z = 0.0f;
  for (int q = 0; q < ks; ++q) z += sums[group * ks + q][lane];
  const int64_t j = n0 + lane / R, i = r0 + lane % R;
  if (j >= p.n || i >= p.rows) return;
  z += p.bias ? to_f32(p.bias[j]) : 0.0f;
  if (p.pre) p.pre[i * p.ldp + j] = from_f32<T>(z);
  z = act_value<T>(z, p.act);
  if (p.residual) z += to_f32(p.residual[i * p.ldr + j]);
  p.y[i * p.ldy + j] = from_f32<T>(z);
}

template <typename T, int VEC, int R>
cudaError_t launch_few_r(const FewParams<T>& p, int ks, cudaStream_t st) {
  const int warps = R == 8 && ks <= 4 ? 4 : kFewWarps;
  const int64_t per = kFewCols * (warps / ks);
  const int64_t blocks = (p.n + per - 1) / per * ((p.rows + R - 1) / R);
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  return launch_after(few_rows_kernel<T, VEC, R>, static_cast<unsigned>(blocks), 32 * warps, 0, st, p, ks);
}
template <typename T, int VEC>
cudaError_t launch_few_v(const FewParams<T>& p, int ks, cudaStream_t st) {
  if (p.rows <= 1) return launch_few_r<T, VEC, 1>(p, ks, st);
  if constexpr (VEC > 1) {
    if (p.rows <= 4) return launch_few_r<T, VEC, 4>(p, ks, st);
  }
  return launch_few_r<T, VEC, 8>(p, ks, st);
}

bool tma_rows(const void* p, int64_t ld, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * bytes % 16 == 0; }

// Whether the rows are few enough, by the times of both (us; w beyond the caches).  Measured, here and on the tensor cores:
// bf16 rows 1, 4, 8, 16 of 512 -> 12288: 3.5, 4.8, 7.9, 14.4 and 8.4, 8.4, 8.4, 7.1; 4096 -> 16384: 23, 29, 48, 77 and
// 41, 36, 37, 26; 16384 -> 512: 4.0, 5.4, 7.3, 13.3 and 45 to 47.  f32 rows 8, 32 and 40: 512 -> 12288 10,
// 21, 27 and 33; 4096 -> 16384 75, 189, 227 and 245; 2007 -> 32552 108 (12), 197, 241 and 251.  bf16 rows off 16-byte
// boundaries: 5 of 2071 -> 48416 87 and 268; 12, 24 and 32 of 2007 -> 32552 109, 158, 202 and 164; 32 of 515 -> 12288 27, 23.
bool few_rows(const Product& g) {
  if (g.m > 40 || !g.a.k_inner || !g.b.k_inner) return false;
  if (g.m <= 4 || g.dtype == kF32) return true;
  const double passes = static_cast<double>((g.m + 7) / 8), values = static_cast<double>(g.n) * g.k;
  const double v = values * 1e-6;
  if (!tma_rows(g.b.p, g.b.ld, 2)) return 6.0 + passes * v * 0.82 < 16.0 + v * 2.35;
  const double depth = static_cast<double>((g.k + 63) / 64), waves = static_cast<double>((g.n + 256 * 76 - 1) / (256 * 76));
  const double products = waves * depth * 0.17, bytes = values * 2 / 5e6;
  return 2.0 + passes * values * 2 / 2.1e6 < 6.0 + (products > bytes ? products : bytes);
}

template <typename T>
cudaError_t launch_few(const Product& g, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  FewParams<T> p{static_cast<const T*>(g.a.p), static_cast<const T*>(g.b.p), g.a.ld, g.b.ld, g.m, g.n, g.k, 0,
                 static_cast<const T*>(g.bias), static_cast<const T*>(g.residual), g.ldr, g.act, static_cast<T*>(g.c), g.ldc,
                 static_cast<T*>(g.pre), g.ldp};
  const bool vec = g.k % kVec == 0 && g.a.ld % kVec == 0 && g.b.ld % kVec == 0 &&
                   (reinterpret_cast<uintptr_t>(g.a.p) | reinterpret_cast<uintptr_t>(g.b.p)) % 16 == 0;
  const int64_t step = 32 * (vec ? kVec : 1);
  // k in parts until there are 16 warps for every SM, each with a step at least
  int ks = 1;
  while (ks < kFewWarps && (g.n + kFewCols - 1) / kFewCols * ks < 16 * ops_sm_count() && g.k > 2 * ks * step) ks *= 2;
  p.k_run = ((g.k + ks - 1) / ks + step - 1) / step * step;
  return vec ? launch_few_v<T, kVec>(p, ks, st) : launch_few_v<T, 1>(p, ks, st);
}

// ---------------------------------------------------------------------------
// dz = dy act'(pre) and its column sums.  A block takes 32 x VEC columns and
// `rows_each` rows, a warp every eighth of them; a column's sums over the
// block go to part[block row][column] and are added in that order by the
// second kernel.
// ---------------------------------------------------------------------------
constexpr int kSumWarps = 8, kSumThreads = 32 * kSumWarps, kSumAhead = 4;

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kSumThreads) slope_sums_kernel(const SlopeSums s, int64_t rows_each) {
  const T* dy = static_cast<const T*>(s.dy);
  const T* pre = static_cast<const T*>(s.pre);
  T* dz = static_cast<T*>(s.dz);
  __shared__ float sums[kSumWarps][32 * VEC];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t col_blocks = (s.n + 32 * VEC - 1) / (32 * VEC);
  const int64_t rb = blockIdx.x / col_blocks;
  const int64_t j0 = (blockIdx.x % col_blocks) * (32 * VEC), j = j0 + lane * VEC;
  const int64_t r1 = min(s.rows, (rb + 1) * rows_each);
  float acc[VEC] = {};
  if (j < s.n) {
    for (int64_t r = rb * rows_each + warp; r < r1; r += kSumWarps * kSumAhead) {
      Raw<T, VEC> v[kSumAhead], z[kSumAhead];
#pragma unroll
      for (int a = 0; a < kSumAhead; ++a) {
        const int64_t i = r + a * kSumWarps;
        if (i < r1) {
          v[a].load_nc(dy + i * s.lddy + j);
          if constexpr (ACT != kActNone) z[a].load_nc(pre + i * s.ldp + j);
        }
      }
#pragma unroll
      for (int a = 0; a < kSumAhead; ++a) {
        const int64_t i = r + a * kSumWarps;
        if (i >= r1) break;
        Vec<T, VEC> t;
        t.set_raw(v[a]);
        if constexpr (ACT != kActNone) {
          Vec<T, VEC> u;
          u.set_raw(z[a]);
#pragma unroll
          for (int c = 0; c < VEC; ++c) t.v[c] *= act_slope<T>(u.v[c], ACT);
          if (dz) {
            t.store(dz + i * s.lddz + j);
            if constexpr (sizeof(T) == 2 && ACT != kActRelu) {  // (relu's dz is dy or 0)
              if (s.rest) {
                Vec<T, VEC> left;
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                  const float lead = to_f32(from_f32<T>(t.v[c]));
                  left.v[c] = fabsf(lead) < INFINITY ? t.v[c] - lead : 0.0f;
                }
                left.store(dz + s.rest + i * s.lddz + j);
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] += t.v[c];
      }
    }
  }
  if (!s.dbias) return;
#pragma unroll
  for (int c = 0; c < VEC; ++c) sums[warp][lane * VEC + c] = acc[c];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * VEC; c += kSumThreads) {
    if (j0 + c >= s.n) break;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) t += sums[w][c];
    s.part[rb * s.n + j0 + c] = t;
  }
}

// A block adds 32 columns' parts, a warp every eighth of them.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) sum_parts_kernel(const float* part, int64_t parts, int64_t n, T* out) {
  __shared__ float sums[kSumWarps][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t j = int64_t(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (j < n) {
#pragma unroll 8
    for (int64_t i = warp; i < parts; i += kSumWarps) t += __ldcg(part + i * n + j);
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && j < n) {
    t = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) t += sums[w][lane];
    out[j] = from_f32<T>(t);
  }
}

template <typename T>
bool slope_vectors(const SlopeSums& s) {
  constexpr int kVec = 16 / sizeof(T);
  const uintptr_t at = reinterpret_cast<uintptr_t>(s.dy) | (s.act != kActNone ? reinterpret_cast<uintptr_t>(s.pre) : 0);
  return at % 16 == 0 && s.lddy % kVec == 0 && s.n % kVec == 0 && (s.act == kActNone || s.ldp % kVec == 0);
}

// Rows of a block: sixteen blocks an SM where there are enough rows, so that the last ones cost little (with four an
// SM a few blocks more than fit at once doubled the time).
int64_t slope_rows_each(int64_t rows, int64_t n) {
  const int64_t col_blocks = (n + 255) / 256;
  const int64_t each = rows * col_blocks / (16 * ops_sm_count());
  const int64_t least = kSumWarps * kSumAhead;
  return each < least ? least : each > 512 ? 512 : (each + least - 1) / least * least;
}

template <typename T, int VEC>
cudaError_t launch_slope_act(const SlopeSums& s, int64_t each, unsigned grid, cudaStream_t st) {
  switch (s.act) {
    case kActRelu: return launch_after(slope_sums_kernel<T, VEC, kActRelu>, grid, kSumThreads, 0, st, s, each);
    case kActGelu: return launch_after(slope_sums_kernel<T, VEC, kActGelu>, grid, kSumThreads, 0, st, s, each);
    case kActSilu: return launch_after(slope_sums_kernel<T, VEC, kActSilu>, grid, kSumThreads, 0, st, s, each);
    default: return launch_after(slope_sums_kernel<T, VEC, kActNone>, grid, kSumThreads, 0, st, s, each);
  }
}

template <typename T>
cudaError_t launch_slope_sums_t(const SlopeSums& s, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const int64_t each = slope_rows_each(s.rows, s.n), parts = slope_sums_parts(s.rows, s.n);
  const bool vec = slope_vectors<T>(s);
  const int64_t wide = 32 * (vec ? kVec : 1);
  const int64_t blocks = parts * ((s.n + wide - 1) / wide);
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const unsigned grid = static_cast<unsigned>(blocks);
  cudaError_t e = vec ? launch_slope_act<T, kVec>(s, each, grid, st) : launch_slope_act<T, 1>(s, each, grid, st);
  if (e == cudaSuccess && s.dbias)
    e = launch_after(sum_parts_kernel<T>, static_cast<unsigned>((s.n + 31) / 32), kSumThreads, 0, st,
                     static_cast<const float*>(s.part), parts, s.n, static_cast<T*>(s.dbias));
  return e;
}

// ---------------------------------------------------------------------------
// The gradients of few rows on the CUDA cores, every product and sum in
// f32: w is read, or dw written, straight from and to memory, where the tensor
// cores' path has to split f32 values into three bf16 parts or to lay out rows
// that TMA cannot address.
//
// dx[r, j] = sum over i of dz[r, i] w[i, j]: a thread keeps a few columns of
// eight rows and goes down its chunk of w's rows, dz's values in shared memory;
// the chunks' sums are added in their order by sum_parts_kernel.  Bound by the
// loads of w (5.0 TB/s at 2 x 4096 x 16384 f32).  f32 columns are read one by
// one, a warp 32 neighbours: any alignment, and in 78 registers faster than 16
// bytes a thread in 120 (12 x 2008 x 32552: 76 and 94 us).
// ---------------------------------------------------------------------------
constexpr int kAcrossThreads = 128, kAcrossDeep = 64;
// A thread's values of a row of w: VEC side by side, or four that lie a block's width apart.
template <typename T, int VEC>
struct Across {
  static constexpr int kCols = VEC;
  Raw<T, VEC> raw;
  __device__ __forceinline__ void load(const T* p, int) { raw.load_nc(p); }
  __device__ __forceinline__ void clear() { raw.clear(); }
  __device__ __forceinline__ Pair pair(int i) const { return raw.pair(i); }
};
template <typename T>
struct Across<T, 1> {
  static constexpr int kCols = 4;
  Raw<T, 1> raw[4];
  __device__ __forceinline__ void load(const T* p, int cols) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < cols) raw[e].load_nc(p + e * kAcrossThreads);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < 4; ++e) raw[e].clear();
  }
  __device__ __forceinline__ Pair pair(int i) const { return Pair::of(to_f32(raw[2 * i].u), to_f32(raw[2 * i + 1].u)); }
};
template <typename T, int VEC, int R>
__global__ void __launch_bounds__(kAcrossThreads) few_rows_across_kernel(const Operand a, const Operand b, int64_t m, int64_t n,
                                                                         int64_t k, int64_t chunk, float* part) {
  using W = Across<T, VEC>;
  constexpr int kPairs = W::kCols / 2, kStep = VEC == 1 ? kAcrossThreads : 1, kAhead = 8;
  __shared__ __align__(16) float as[kAcrossDeep][R];
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned passes = static_cast<unsigned>((m + R - 1) / R);  // side by side, so that w is in L2 for all but the first
  const int64_t j = int64_t(blockIdx.x / passes) * kAcrossThreads * W::kCols + threadIdx.x * (VEC == 1 ? 1 : VEC);
  const int64_t k0 = int64_t(blockIdx.y) * chunk, k1 = min(k, k0 + chunk), r0 = blockIdx.x % passes * R;
  const T* ap = static_cast<const T*>(a.p) + r0 * a.ld;
  const T* bp = static_cast<const T*>(b.p) + j;
  const int cols = j >= n ? 0 : VEC > 1 ? VEC : static_cast<int>(min(int64_t(4), (n - j + kStep - 1) / kStep));
  Pair two[R][kPairs];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) two[r][i] = Pair::of(0.0f, 0.0f);
  for (int64_t i0 = k0; i0 < k1; i0 += kAcrossDeep) {
    __syncthreads();
    for (int e = threadIdx.x; e < kAcrossDeep * R; e += kAcrossThreads) {
      const int i = e % kAcrossDeep, r = e / kAcrossDeep;
      float v = 0.0f;
      if (i0 + i < k1 && r0 + r < m) {
        v = to_f32(ap[r * a.ld + i0 + i]);
        if (a.rest) v += to_f32(ap[a.rest + r * a.ld + i0 + i]);
      }
      as[i][r] = v;
    }
    __syncthreads();
    const int deep = static_cast<int>(min(int64_t(kAcrossDeep), k1 - i0));
    if (!cols) continue;
    for (int i = 0; i < deep; i += kAhead) {
      W v[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        v[e].clear();
        if (i + e < deep) v[e].load(bp + (i0 + i + e) * b.ld, cols);
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (i + e >= deep) break;
        Pair w[kPairs];
#pragma unroll
        for (int q = 0; q < kPairs; ++q) w[q] = v[e].pair(q);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = as[i + e][r];
#pragma unroll
          for (int q = 0; q < kPairs; ++q) two[r][q].fma(Pair::of(f, f), w[q]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r0 + r >= m) break;
    float* dst = part + (int64_t(blockIdx.y) * m + r0 + r) * n + j;
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      float lo, hi;
      two[r][q].get(&lo, &hi);
      if (2 * q < cols) dst[2 * q * kStep] = lo;
      if (2 * q + 1 < cols) dst[(2 * q + 1) * kStep] = hi;
    }
  }
}

// dw[i, j] = sum over few r of dz[r, i] x[r, j]: a thread makes 8 x 4 results,
// its four columns 64 apart, so that a warp writes 32 neighbours whatever the
// rows' alignment.  Bound by the stores of dw with up to some 8 rows (5.9 TB/s
// at 2 x 4096 x 16384 f32), by the products above.
constexpr int kOuterRows = 32, kOuterCols = 256, kOuterThreads = 256, kOuterMost = 32;
template <typename T>
__global__ void __launch_bounds__(kOuterThreads) few_outer_kernel(const Operand a, const Operand b, int64_t m, int64_t n, int k, T* c,
                                                                  int64_t ldc, int64_t col_tiles) {
  __shared__ __align__(16) float as[kOuterMost][kOuterRows];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t i0 = blockIdx.x / col_tiles * kOuterRows, j0 = blockIdx.x % col_tiles * kOuterCols;
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  const T* ap = static_cast<const T*>(a.p);
  const T* bp = static_cast<const T*>(b.p);
  for (int e = threadIdx.x; e < k * kOuterRows; e += kOuterThreads) {
    const int i = e % kOuterRows, r = e / kOuterRows;
    float v = 0.0f;
    if (i0 + i < m) {
      v = to_f32(ap[r * a.ld + i0 + i]);
      if (a.rest) v += to_f32(ap[a.rest + r * a.ld + i0 + i]);
    }
    as[r][i] = v;
  }
  __syncthreads();
  Pair acc[4][4];  // two rows in each
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = Pair::of(0.0f, 0.0f);
#pragma unroll 4
  for (int r = 0; r < k; ++r) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t j = j0 + e * 64 + tx;
      x[e] = j < n ? to_f32(__ldg(bp + r * b.ld + j)) : 0.0f;
    }
    const float4 z0 = *reinterpret_cast<const float4*>(&as[r][ty * 8]), z1 = *reinterpret_cast<const float4*>(&as[r][ty * 8 + 4]);
    const Pair z[4] = {Pair::of(z0.x, z0.y), Pair::of(z0.z, z0.w), Pair::of(z1.x, z1.y), Pair::of(z1.z, z1.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Pair xx = Pair::of(x[e], x[e]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][e].fma(z[i], xx);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = i0 + ty * 8 + i;
    if (row >= m) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t j = j0 + e * 64 + tx;
      float lo, hi;
      acc[i / 2][e].get(&lo, &hi);
      if (j < n) c[row * ldc + j] = from_f32<T>(i % 2 ? hi : lo);
    }
  }
}

bool plain_product(const Product& g) { return !g.bias && !g.residual && !g.pre && g.act == kActNone; }

// Whether dx is formed by passes over w.  Measured (us) for rows x inner x outer, here and on the tensor cores: f32
// 3 x 512 x 12288 14 and 66, 2 x 4096 x 16384 54 and 242, 12 x 2007 x 32552 76 and 255, 32 x 2007 x 32552 146 and 258; bf16
// off 16-byte boundaries 5 x 2071 x 48416 83 and 278, 12, 24 and 32 x 2007 x 32552 85, 124, 164 and 168; bf16 that TMA
// addresses 2 x 4096 x 16384 35 and 42, 8 x 512 x 65536 28 and 41, 16 x 4096 x 16384 72 and 35.
bool few_across(const Product& g) {
  if (!plain_product(g) || !g.a.k_inner || g.b.k_inner || g.ldc != g.n || g.m * g.n / 32 >= INT32_MAX) return false;
  if (g.dtype == kF32) return g.m <= 48;
  return tma_rows(g.b.p, g.b.ld, 2) ? g.m <= 8 && g.n % 8 == 0 : g.m <= 32;
}
// Whether dw is formed from few rows, by the estimated times (us) of the two paths.  Measured, here and on the tensor cores:
// f32 2, 8, 16 and 32 x 4096 x 16384 46, 57, 85, 128 and 75; 12 and 32 x 2007 x 32552 80, 134 and 170; 32 x 512 x 12288 16
// and 21; bf16 5 x 2071 x 48416 78 and 102, 12 x 2007 x 32552 72 and 67, 2 x 4096 x 16384 39 and 28, 8 and 32 x 512 x 12288
// 11, 17 and 15, 30 x 300 x 5000 11 and 19.
bool few_outer(const Product& g) {
  if (!plain_product(g) || g.a.k_inner || g.b.k_inner || g.k > kOuterMost) return false;
  const double values = static_cast<double>(g.m) * g.n * 1e-6, k = static_cast<double>(g.k);
  if (g.dtype == kF32) return 5.0 + values * (0.6 + 0.04 * k) < 16.0 + values * (tma_rows(g.c, g.ldc, 4) ? 0.88 : 2.37);
  const double here = 4.0 + values * (0.5 + 0.047 * k);
  const bool tma = tma_rows(g.a.p, g.a.ld, 2) && tma_rows(g.b.p, g.b.ld, 2) && tma_rows(g.c, g.ldc, 2);
  return here < (tma ? 14.0 + values * 0.195 : 12.5 + values * 0.83);
}
constexpr int kAcrossRows = 8;
bool across_vec(const Product& g) { return g.dtype != kF32 && tma_rows(g.b.p, g.b.ld, 2) && g.n % 8 == 0; }
int64_t across_tiles(const Product& g) {
  const int64_t wide = kAcrossThreads * (across_vec(g) ? 8 : 4);
  return (g.n + wide - 1) / wide * ((g.m + kAcrossRows - 1) / kAcrossRows);
}
// Chunks of w's rows, of 64 at least: as many blocks as the SMs hold at once (12 x 2007 x 32552 f32, 4, 6 and 12 blocks an
// SM: 108, 76 and 79 us; 2 x 4096 x 16384 bf16, whose threads hold eight columns: 36, 42 and 38).
int64_t across_chunks(const Product& g) {
  int64_t chunks = (across_vec(g) ? 4 : 6) * ops_sm_count() / across_tiles(g);
  const int64_t most = (g.k + kAcrossDeep - 1) / kAcrossDeep;
  chunks = chunks > most ? most : chunks;
  return chunks < 1 ? 1 : chunks;
}
template <typename T>
cudaError_t launch_across(const Product& g, Scratch& sc, cudaStream_t st) {
  const int64_t chunks = across_chunks(g);
  float* part = sc.take<float>(chunks * g.m * g.n);
  const int64_t chunk = (g.k + chunks - 1) / chunks;
  if (across_tiles(g) > INT32_MAX) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(across_tiles(g)), static_cast<unsigned>((g.k + chunk - 1) / chunk));
  cudaError_t e;
  if constexpr (sizeof(T) == 2) {
    e = across_vec(g) ? launch_after(few_rows_across_kernel<T, 8, kAcrossRows>, grid, kAcrossThreads, 0, st, g.a, g.b, g.m, g.n, g.k,
                                     chunk, part)
                      : launch_after(few_rows_across_kernel<T, 1, kAcrossRows>, grid, kAcrossThreads, 0, st, g.a, g.b, g.m, g.n, g.k,
                                     chunk, part);
  } else {
    e = launch_after(few_rows_across_kernel<T, 1, kAcrossRows>, grid, kAcrossThreads, 0, st, g.a, g.b, g.m, g.n, g.k, chunk, part);
  }
  if (e != cudaSuccess) return e;
  return launch_after(sum_parts_kernel<T>, static_cast<unsigned>((g.m * g.n + 31) / 32), kSumThreads, 0, st,
                      static_cast<const float*>(part), int64_t(grid.y), g.m * g.n, static_cast<T*>(g.c));
}
template <typename T>
cudaError_t launch_outer(const Product& g, cudaStream_t st) {
  const int64_t col_tiles = (g.n + kOuterCols - 1) / kOuterCols, blocks = col_tiles * ((g.m + kOuterRows - 1) / kOuterRows);
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  return launch_after(few_outer_kernel<T>, static_cast<unsigned>(blocks), kOuterThreads, 0, st, g.a, g.b, g.m, g.n,
                      static_cast<int>(g.k), static_cast<T*>(g.c), g.ldc, col_tiles);
}

}  // namespace

int64_t slope_sums_parts(int64_t rows, int64_t n) {
  const int64_t each = slope_rows_each(rows, n);
  return (rows + each - 1) / each;
}

cudaError_t launch_slope_sums(const SlopeSums& s, cudaStream_t st) {
  return s.dtype == kF32 ? launch_slope_sums_t<float>(s, st) : launch_slope_sums_t<__nv_bfloat16>(s, st);
}

size_t product_scratch_bytes(const Product& g) {
  if (few_rows(g) || few_outer(g)) return 0;
  if (few_across(g)) {
    Scratch sc;
    sc.take<float>(across_chunks(g) * g.m * g.n);
    return sc.used();
  }
  return mma_scratch_bytes(g);
}

cudaError_t launch_product(const Product& g, Scratch& sc, const Words& words, cudaStream_t st) {
  const bool f32 = g.dtype == kF32;
  if (few_rows(g)) return f32 ? launch_few<float>(g, st) : launch_few<__nv_bfloat16>(g, st);
  if (few_outer(g)) return f32 ? launch_outer<float>(g, st) : launch_outer<__nv_bfloat16>(g, st);
  if (few_across(g)) return f32 ? launch_across<float>(g, sc, st) : launch_across<__nv_bfloat16>(g, sc, st);
  static std::atomic<int> calls{0};
  const int call = f32 || g.a.rest ? 1 + (calls.fetch_add(1) & 0x3fffffff) : 0;
  return launch_mma(g, sc, words, call, st);
}

cudaError_t launch_simt(const Product& g, const int* marks, int call, cudaStream_t st) { return launch_simt_t(g, marks, call, st); }

}  // namespace tk
